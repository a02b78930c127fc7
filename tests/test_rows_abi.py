"""Argument rules of the 8-bit row operators: each answers before any CUDA work. Runs without a GPU."""
import ctypes

import pytest
import torch

import weight_only_quantized_wq4_gb300 as wq4

P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(10)]      # aligned stand-ins, never dereferenced
MIS = ctypes.c_void_p(0x10001)
HALF = ctypes.c_void_p(0x10008)
REFUSED = (wq4.ERR_INVALID, wq4.ERR_ALIGN, wq4.ERR_UNSUPPORTED)


@pytest.fixture(scope="module")
def clib():
    wq4.build()
    return wq4.load_library()


def test_norm_rules(clib):
    def call(X=P[0], ldx=256, R=P[1], ldr=256, w=P[2], T=4, D=256, eps=1e-5, dt=0, Ro=P[3], ldro=256, Y=P[4], ldy=256,
             Q=P[5], ldq=256, s=P[6], lds=4):
        return clib.wq4_add_rmsnorm_quant(X, ldx, R, ldr, w, T, D, eps, dt, Ro, ldro, Y, ldy, Q, ldq, s, lds, None)

    assert call() not in REFUSED                                   # valid (fails later, without a GPU)
    assert call(R=None, Ro=None) not in REFUSED
    assert call(Q=None, s=None) not in REFUSED and call(Y=None) not in REFUSED and call(Ro=None) not in REFUSED
    assert call(X=ctypes.c_void_p(0x10002), ldx=259) not in REFUSED   # 2-byte rows are allowed
    assert call(T=0, X=None, R=None, w=None, Ro=None, Y=None, Q=None, s=None) == wq4.OK
    for bad in (dict(T=-1), dict(D=0), dict(dt=2), dict(dt=-1), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(X=None), dict(w=None), dict(R=None), dict(Y=None, Q=None, s=None),
                dict(Q=None), dict(s=None), dict(ldx=255), dict(ldr=255), dict(ldro=255), dict(ldy=255),
                dict(ldq=255), dict(lds=3)):
        assert call(**bad) == wq4.ERR_INVALID, bad
    for bad in (dict(X=MIS), dict(R=MIS), dict(w=MIS), dict(Ro=MIS), dict(Y=MIS), dict(Q=HALF), dict(s=HALF),
                dict(ldq=264), dict(lds=5)):
        assert call(**bad) == wq4.ERR_ALIGN, bad
    assert call(D=32769, ldx=40000, ldr=40000, ldro=40000, ldy=40000, ldq=40000) == wq4.ERR_UNSUPPORTED


def test_gated_rules(clib):
    def call(X=P[0], ldx=512, T=4, D=256, dt=0, Q=P[5], ldq=256, s=P[6], lds=4):
        return clib.wq4_silu_mul_quant(X, ldx, T, D, dt, Q, ldq, s, lds, None)

    assert call() not in REFUSED
    assert call(T=0, X=None, Q=None, s=None) == wq4.OK
    for bad in (dict(T=-1), dict(D=0), dict(dt=2), dict(X=None), dict(Q=None), dict(s=None), dict(ldx=511),
                dict(ldq=255), dict(lds=3)):
        assert call(**bad) == wq4.ERR_INVALID, bad
    for bad in (dict(X=MIS), dict(Q=HALF), dict(s=HALF), dict(ldq=257), dict(lds=6)):
        assert call(**bad) == wq4.ERR_ALIGN, bad
    assert call(D=(1 << 24) + 1, ldx=1 << 26, ldq=1 << 26) == wq4.ERR_UNSUPPORTED
    assert call(T=1 << 30, D=1 << 20, ldx=1 << 21, ldq=1 << 20, lds=1 << 30) == wq4.ERR_UNSUPPORTED


def test_product_rules(clib):
    def call(X=P[0], ldx=256, sx=P[1], ldsx=8, W=P[2], ldw=256, sw=P[3], ldsw=2, Y=P[4], ldy=384, M=5, N=384, K=256, dt=0):
        return clib.wq4_block_mm(X, ldx, sx, ldsx, W, ldw, sw, ldsw, Y, ldy, M, N, K, dt, None)

    assert call() not in REFUSED and call(dt=2) not in REFUSED
    assert call(N=3, K=16) not in REFUSED
    assert call(M=0, X=None, sx=None, W=None, sw=None, Y=None) == wq4.OK
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(dt=3), dict(dt=-1), dict(X=None), dict(sx=None), dict(W=None),
                dict(sw=None), dict(Y=None), dict(ldx=240), dict(ldw=240), dict(ldsx=4), dict(ldsw=1), dict(ldy=383)):
        assert call(**bad) == wq4.ERR_INVALID, bad
    for bad in (dict(X=HALF), dict(W=HALF), dict(sx=HALF), dict(sw=ctypes.c_void_p(0x10002)), dict(Y=MIS),
                dict(Y=ctypes.c_void_p(0x10002), dt=2), dict(ldx=264), dict(ldw=264), dict(ldsx=9)):
        assert call(**bad) == wq4.ERR_ALIGN, bad
    assert call(K=250) == wq4.ERR_UNSUPPORTED
    assert call(ldw=1 << 40) == wq4.ERR_UNSUPPORTED


def test_logprobs_rules(clib):
    def call(x=P[0], ld=1000, tok=P[1], T=3, V=1000, dt=2, k=5, lp=P[2], ent=P[3], ids=P[4], tlp=P[5]):
        return clib.wq4_token_logprobs(x, ld, tok, T, V, dt, k, lp, ent, ids, tlp, None)

    assert call() not in REFUSED
    assert call(tok=None, lp=None) not in REFUSED and call(ent=None) not in REFUSED
    assert call(k=0, ids=None, tlp=None) not in REFUSED
    assert call(x=ctypes.c_void_p(0x10002), dt=0, ld=1001) not in REFUSED
    assert call(T=0, x=None, tok=None, lp=None, ent=None, ids=None, tlp=None) == wq4.OK
    for bad in (dict(T=-1), dict(V=0), dict(dt=3), dict(k=-1), dict(V=4), dict(x=None), dict(ld=999), dict(tok=None),
                dict(lp=None), dict(ids=None), dict(tlp=None), dict(k=0), dict(k=0, ids=None),
                dict(k=0, ids=None, tlp=None, tok=None, lp=None, ent=None)):
        assert call(**bad) == wq4.ERR_INVALID, bad
    for bad in (dict(x=ctypes.c_void_p(0x10002)), dict(x=MIS, dt=0), dict(tok=ctypes.c_void_p(0x10004)), dict(lp=MIS),
                dict(ent=MIS), dict(ids=MIS), dict(tlp=MIS)):
        assert call(**bad) == wq4.ERR_ALIGN, bad
    assert call(k=33) == wq4.ERR_UNSUPPORTED
    assert call(V=(1 << 30) + 1, ld=1 << 31) == wq4.ERR_UNSUPPORTED


def test_binding_refuses_cpu_tensors_and_wrong_shapes(clib):
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    for call in (lambda: wq4.add_rmsnorm_quant(x, x[0]), lambda: wq4.silu_mul_quant(x),
                 lambda: wq4.silu_mul_quant(x[0]), lambda: wq4.add_rmsnorm_quant(x.float(), x[0]),
                 lambda: wq4.block_mm(x, x, x, x), lambda: wq4.token_logprobs(x)):
        with pytest.raises(ValueError):
            call()


def test_quant_row_buffers_are_padded():
    q, s = wq4.alloc_quant_rows(5, 200, device="cpu")
    assert q.shape == (5, 200) and q.stride() == (208, 1) and q.dtype == torch.float8_e4m3fn
    assert s.shape == (2, 5) and s.stride() == (8, 1) and s.dtype == torch.float32
