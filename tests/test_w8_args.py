"""Argument checks and host-side queries of lq_quant_i8, lq_norm_residual and lq_gemm_i8. No GPU
is used: every call below returns before any CUDA work."""
import ctypes

import pytest
import torch

import fractional_bit_weight_b200 as lq
from fractional_bit_weight_b200 import build as lqbuild

FAKE = 0x10000      # aligned, never dereferenced
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    lqbuild.build()
    return lq.lib()


def test_row_bytes(L):
    assert [lq.i8_row_bytes(k) for k in (1, 15, 16, 17, 4096, 2 ** 31 - 1)] == \
        [16, 16, 16, 32, 4096, 2 ** 31]
    assert lq.i8_row_bytes(0) == -1


def test_routes(L):
    assert lq.gemm_i8_route(1, 4096, 4096) == lq.I8_ROUTE_GEMV
    assert lq.gemm_i8_route(2048, 8192, 28672) == lq.I8_ROUTE_PAIR
    assert lq.gemm_i8_route(128, 4096, 4096) == lq.I8_ROUTE_TC
    assert lq.gemm_i8_route(8, 28672, 8192) == lq.I8_ROUTE_GEMV
    assert lq.gemm_i8_route(1, 8192, 28672) in (lq.I8_ROUTE_TC, lq.I8_ROUTE_PAIR)
    assert lq.gemm_i8_route(16, 4096, 4096) == lq.I8_ROUTE_GEMV
    assert lq.gemm_i8_route(16, 8192, 28672) in (lq.I8_ROUTE_TC, lq.I8_ROUTE_PAIR)
    assert lq.gemm_i8_route(17, 64, 64) == lq.I8_ROUTE_TC
    assert lq.gemm_i8_route(20, 28672, 1024) == lq.I8_ROUTE_SPLIT
    assert lq.gemm_i8_route(1, 28672, 1024) == lq.I8_ROUTE_SPLIT
    assert lq.gemm_i8_route(1, 14336, 1024) == lq.I8_ROUTE_GEMV
    assert lq.gemm_i8_route(2**30, 64, 64) == lq.I8_ROUTE_TC
    assert lq.gemm_i8_route(2**30, 64, 2**30) in (lq.I8_ROUTE_TC, lq.I8_ROUTE_PAIR)
    for bad in ((0, 64, 64), (1, 0, 64), (1, 64, 0), (1, 131072, 64), (2 ** 30 + 1, 64, 64),
                (1, 64, 2 ** 30 + 1)):
        assert lq.gemm_i8_route(*bad) == -1


def quant(L, **kw):
    a = dict(x=FAKE, dt=2, rows=4, K=64, ld=64, T=None, q=FAKE, s=FAKE, v=None)
    a.update(kw)
    return L.lq_quant_i8(a["x"], a["dt"], a["rows"], a["K"], a["ld"], a["T"], a["q"], a["s"],
                         a["v"], None)


def test_quant_arguments(L):
    for kw in (dict(x=None), dict(q=None), dict(s=None), dict(dt=3), dict(rows=-1), dict(K=0),
               dict(ld=63), dict(x=FAKE + 1), dict(q=FAKE + 8), dict(s=FAKE + 2),
               dict(v=FAKE + 1), dict(T=ctypes.byref(lq.WhitenDesc(None, None, 3))),
               dict(T=ctypes.byref(lq.WhitenDesc(None, None, 128)))):
        assert quant(L, **kw) == lq.LQ_EINVAL, kw
        assert L.lq_last_error()
    assert quant(L, K=65537, ld=65537) == lq.LQ_EUNSUPPORTED
    assert quant(L, K=8192, ld=8192, T=ctypes.byref(lq.WhitenDesc(None, None, 8192))) == \
        lq.LQ_EUNSUPPORTED
    assert quant(L, rows=0) == lq.LQ_OK
    assert quant(L, rows=0, x=None, q=None, s=None) == lq.LQ_OK


def boundary(L, **kw):
    a = dict(h=FAKE, hdt=0, ldh=64, r=FAKE, rdt=2, ldr=64, rows=4, K=64, post=None, gate=None,
             ro=FAKE, pre=None, n=FAKE, ndt=2, T=None, q=None, qs=None)
    a.update(kw)
    ref = lambda d: None if d is None else ctypes.byref(d)  # noqa: E731
    return L.lq_norm_residual(a["h"], a["hdt"], a["ldh"], a["r"], a["rdt"], a["ldr"], a["rows"],
                              a["K"], ref(a["post"]), ref(a["gate"]), 1.0, 1.0, a["ro"],
                              ref(a["pre"]), a["n"], a["ndt"], ref(a["T"]), a["q"], a["qs"], None)


def test_boundary_arguments(L):
    norm, gate = lq.NormDesc, lq.GateDesc
    for kw in (dict(h=None), dict(hdt=9), dict(rdt=9), dict(ndt=9), dict(rows=-1), dict(K=0),
               dict(ldh=63), dict(ldr=60), dict(ro=None, n=None), dict(q=FAKE), dict(qs=FAKE),
               dict(h=FAKE + 2), dict(r=FAKE + 1), dict(ro=FAKE + 1), dict(n=FAKE + 1),
               dict(q=FAKE + 4, qs=FAKE), dict(q=FAKE, qs=FAKE + 1),
               dict(post=norm(0, 1e-6, None, None, 0)), dict(pre=norm(3, 1e-6, None, None, 0)),
               dict(pre=norm(1, -1e-6, None, None, 0)), dict(pre=norm(1, NAN, None, None, 0)),
               dict(pre=norm(1, float("inf"), None, None, 0)),
               dict(post=norm(1, 1e-6, FAKE, None, 5)), dict(post=norm(1, 1e-6, FAKE + 2, None, 0)),
               dict(post=norm(2, 1e-6, None, FAKE + 1, 1)), dict(gate=gate(None, 0, 64, 1)),
               dict(gate=gate(FAKE, 4, 64, 1)), dict(gate=gate(FAKE, 0, 63, 1)),
               dict(gate=gate(FAKE, 0, 64, 0)), dict(gate=gate(FAKE + 2, 0, 64, 1)),
               dict(q=FAKE, qs=FAKE, T=lq.WhitenDesc(None, None, 128))):
        assert boundary(L, **kw) == lq.LQ_EINVAL, kw
        assert L.lq_last_error()
    assert boundary(L, K=65544, ldh=65544, ldr=65544) == lq.LQ_EUNSUPPORTED
    assert boundary(L, rows=0) == lq.LQ_OK


def gemm(L, **kw):
    a = dict(xq=FAKE, xs=FAKE, batch=4, wq=FAKE, ws=FAKE, b=None, K=64, N=32, y=FAKE, dt=0,
             w=FAKE, wb=256, route=-1)
    a.update(kw)
    return L.lq_gemm_i8(a["xq"], a["xs"], a["batch"], a["wq"], a["ws"], a["b"], a["K"], a["N"],
                        a["y"], a["dt"], a["w"], a["wb"], a["route"], None)


def test_gemm_arguments(L):
    for kw in (dict(xq=None), dict(xs=None), dict(wq=None), dict(ws=None), dict(y=None),
               dict(w=None), dict(batch=-1), dict(N=-1), dict(K=0), dict(dt=3), dict(route=4),
               dict(route=-2), dict(xq=FAKE + 8), dict(wq=FAKE + 4), dict(xs=FAKE + 2),
               dict(ws=FAKE + 1), dict(b=FAKE + 2), dict(y=FAKE + 2), dict(y=FAKE + 1, dt=2),
               dict(w=FAKE + 128), dict(wb=255)):
        assert gemm(L, **kw) == lq.LQ_EINVAL, kw
        assert L.lq_last_error()
    assert gemm(L, K=131072) == lq.LQ_EUNSUPPORTED
    assert gemm(L, N=2 ** 30 + 1) == lq.LQ_EUNSUPPORTED
    assert gemm(L, batch=2 ** 30 + 1) == lq.LQ_EUNSUPPORTED
    assert gemm(L, batch=17, route=lq.I8_ROUTE_GEMV) == lq.LQ_EUNSUPPORTED
    assert gemm(L, batch=0) == lq.LQ_OK
    assert gemm(L, N=0) == lq.LQ_OK


def test_host_tensors_are_refused():
    x = torch.randn(2, 64)
    q = torch.zeros(2, 64, dtype=torch.int8)
    s = torch.ones(2)
    for call in (lambda: lq.quant_i8(x), lambda: lq.norm_residual(x), lambda: lq.norm_residual_i8(x),
                 lambda: lq.gemm_i8(q, s, q, s), lambda: lq.Norm("rms", torch.ones(64))):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="norm kind"):
        lq.Norm("batch")
