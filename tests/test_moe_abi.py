"""Argument checks of the mixture-of-experts entry points; no GPU: every
rejection happens before the device is touched."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "quantized_matmul_amd", "libqlin.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libqlin.so not built")

INVALID, UNSUPPORTED = 1, 2
F32, F16, BF16, U8 = 0, 1, 2, 3
P = ctypes.c_void_p(0x1000)   # never dereferenced: validation rejects first
ODD = ctypes.c_void_p(0x1001)


@pytest.fixture(scope="module")
def lib():
    from quantized_matmul_amd import _binding
    return _binding.load_library()


def err(lib):
    return lib.qlin_last_error().decode()


def test_header_functions_are_exported(lib):
    text = open(os.path.join(ROOT, "include", "qlin.h")).read()
    names = set(re.findall(r"\b(qlin_[a-z0-9_]+)\s*\(", text))
    assert names >= {"qlin_moe_route", "qlin_moe_route_grad", "qlin_mxfp4_matmul", "qlin_gather_mxfp4_matmul",
                     "qlin_mxfp4_matmul_workspace_bytes", "qlin_gather_mxfp4_matmul_workspace_bytes",
                     "qlin_moe_combine", "qlin_moe_combine_grad"}
    for n in names:
        assert hasattr(lib, n), n


def caller(f, base):
    return lambda **kw: f(*dict(base, **kw).values())


def test_route_rejects(lib):
    call = caller(lib.qlin_moe_route, dict(x=P, dt=BF16, T=4, E=64, k=8, bias=None, score=b"softmax", renorm=1,
                                           scale=1.0, groups=1, kept=1, top=1, w=P, e=P, st=None))
    for bad in (dict(dt=U8), dict(E=0), dict(E=1025), dict(k=0), dict(k=65), dict(E=4, k=5), dict(T=-1),
                dict(score=b"tanh"), dict(score=None), dict(scale=float("inf")), dict(scale=1e39),
                dict(groups=5), dict(groups=0), dict(groups=8, kept=9), dict(groups=8, kept=0),
                dict(groups=8, kept=2, top=3), dict(groups=64, kept=8, top=2), dict(groups=16, kept=1, k=8),
                dict(x=None), dict(w=None), dict(e=None), dict(x=ODD), dict(dt=F32, x=ctypes.c_void_p(0x1002)),
                dict(bias=ctypes.c_void_p(0x1002)), dict(w=ODD), dict(e=ODD)):
        assert call(**bad) == INVALID, bad
        assert err(lib)
    assert call(T=1 << 31) == UNSUPPORTED
    assert call(T=0, x=None, w=None, e=None) == 0
    assert err(lib) == ""


def test_route_grad_rejects(lib):
    call = caller(lib.qlin_moe_route_grad, dict(x=P, dt=F32, T=4, E=64, k=8, e=P, g=P, score=b"sigmoid", renorm=1,
                                                scale=1.0, out=P, st=None))
    for bad in (dict(dt=U8), dict(E=2000), dict(k=0), dict(T=-1), dict(score=b""), dict(scale=float("nan")),
                dict(x=None), dict(e=None), dict(g=None), dict(out=None), dict(x=ODD), dict(e=ODD), dict(g=ODD),
                dict(out=ODD)):
        assert call(**bad) == INVALID, bad
    assert call(T=0, x=None, e=None, g=None, out=None) == 0


def test_product_rejects(lib):
    need = lib.qlin_mxfp4_matmul_workspace_bytes(40, 1024, 4096, BF16)
    assert need > 0
    call = caller(lib.qlin_mxfp4_matmul, dict(x=P, xdt=BF16, xs=None, act=b"none", M=40, K=1024, wq=P, ws=P, N=4096,
                                              work=P, nb=need, y=P, ydt=BF16, st=None))
    for bad in (dict(xdt=7), dict(ydt=U8), dict(act=b"gelu"), dict(M=-1), dict(K=0), dict(K=48), dict(N=0),
                dict(x=None), dict(wq=None), dict(ws=None), dict(y=None), dict(xs=P), dict(xdt=U8),
                dict(xdt=U8, xs=P, act=b"swiglu"), dict(xdt=U8, xs=P, x=ctypes.c_void_p(0x1008)), dict(x=ODD),
                dict(wq=ctypes.c_void_p(0x1004)), dict(y=ODD), dict(work=None), dict(nb=need - 1),
                dict(work=ctypes.c_void_p(0x1008))):
        assert call(**bad) == INVALID, bad
        assert err(lib)
    assert call(K=1 << 23) == UNSUPPORTED
    # more work-items than one launch takes, by the streaming and by the tiled kernel
    assert call(M=1, K=32, N=(1 << 31) - 1, work=None, nb=0) == UNSUPPORTED and "launch" in err(lib)
    assert call(M=(1 << 31) - 1, K=32, N=1 << 20, nb=1 << 60) == UNSUPPORTED and "launch" in err(lib)
    assert call(M=0, x=None, wq=None, ws=None, y=None, work=None, nb=0) == 0
    # a few rows need none: they are quantized inside the product, or given as codes
    assert lib.qlin_mxfp4_matmul_workspace_bytes(4, 128, 64, BF16) == 0
    assert lib.qlin_mxfp4_matmul_workspace_bytes(4, 128, 64, U8) == 0
    assert lib.qlin_mxfp4_matmul_workspace_bytes(4, 100, 64, BF16) == 0


def test_gather_rejects(lib):
    size = lib.qlin_gather_mxfp4_matmul_workspace_bytes
    assert size(4, 8, 128, 16, 64, BF16) == 0    # hardly two rows share an expert: no plan
    assert size(4, 32, 128, 16, 64, BF16) == 0   # or W is so small that each reads it for itself
    need = size(4, 32, 1024, 16, 2048, BF16)
    assert need > 0
    call = caller(lib.qlin_gather_mxfp4_matmul, dict(x=P, xdt=BF16, xs=None, act=None, B=4, K=1024, wq=P, ws=P, E=16,
                                                     N=2048, e=P, R=32, work=P, nb=need, y=P, ydt=F32, st=None))
    for bad in (dict(R=17), dict(B=0), dict(B=-4), dict(R=-8), dict(E=0), dict(e=None), dict(K=33), dict(nb=need - 1),
                dict(work=None), dict(e=ODD), dict(act=b"relu"), dict(ydt=U8)):
        assert call(**bad) == INVALID, bad
        assert err(lib)
    assert call(E=8001) == UNSUPPORTED
    assert call(B=1 << 30, R=1 << 31) == UNSUPPORTED
    assert call(B=(1 << 31) - 1, R=(1 << 31) - 1) == UNSUPPORTED
    assert call(B=0, R=0, x=None, e=None, work=None, nb=0) == 0


def test_combine_rejects(lib):
    call = caller(lib.qlin_moe_combine, dict(h=P, dt=F16, T=4, k=8, D=64, w=P, e=None, y=P, st=None))
    for bad in (dict(dt=U8), dict(T=-1), dict(k=0), dict(D=0), dict(h=None), dict(w=None), dict(y=None), dict(h=ODD),
                dict(w=ODD), dict(e=ODD), dict(y=ODD)):
        assert call(**bad) == INVALID, bad
    assert call(T=1 << 20, k=1 << 20) == UNSUPPORTED
    assert call(T=0, h=None, w=None, y=None) == 0
    call = caller(lib.qlin_moe_combine_grad, dict(gy=P, h=P, dt=BF16, T=4, k=8, D=64, w=P, e=None, gh=P, gw=P, st=None))
    for bad in (dict(dt=U8), dict(T=-1), dict(k=0), dict(D=0), dict(gy=None), dict(h=None), dict(w=None), dict(gh=None),
                dict(gw=None), dict(gy=ODD), dict(gw=ODD), dict(gh=ODD)):
        assert call(**bad) == INVALID, bad
    assert call(T=0, gy=None, h=None, w=None, gh=None, gw=None) == 0


def test_scales_at_odd_addresses_are_no_limit(lib):
    """A weight whose scales are not 16-byte aligned is refused no sooner and asks for no more than another."""
    base = dict(x=P, xdt=BF16, xs=None, act=None, B=2048, K=16384, wq=P, ws=P, E=8, N=4096, e=P, R=16384, work=None,
                nb=0, y=P, ydt=BF16, st=None)
    need = lib.qlin_gather_mxfp4_matmul_workspace_bytes(2048, 16384, 16384, 8, 4096, BF16)
    for scales in (P, ODD, ctypes.c_void_p(0x1008)):
        assert caller(lib.qlin_gather_mxfp4_matmul, base)(ws=scales) == INVALID
        assert f"workspace of {need} bytes" in err(lib)
    base = dict(x=P, xdt=BF16, xs=None, act=None, M=1 << 20, K=16384, wq=P, ws=P, N=16384, work=None, nb=0, y=P,
                ydt=BF16, st=None)
    need = lib.qlin_mxfp4_matmul_workspace_bytes(1 << 20, 16384, 16384, BF16)
    for scales in (P, ODD, ctypes.c_void_p(0x1008)):
        assert caller(lib.qlin_mxfp4_matmul, base)(ws=scales) == INVALID
        assert f"workspace of {need} bytes" in err(lib)


def test_limits_that_the_header_states(lib):
    """No product within them is refused; x of 2^32 values by experts is, unless index rows are no more than experts."""
    dense = caller(lib.qlin_mxfp4_matmul, dict(x=P, xdt=BF16, xs=None, act=None, M=0, K=0, wq=P, ws=P, N=0, work=None,
                                               nb=0, y=P, ydt=BF16, st=None))
    gather = caller(lib.qlin_gather_mxfp4_matmul, dict(x=P, xdt=BF16, xs=None, act=None, B=0, K=0, wq=P, ws=P, E=0,
                                                       N=0, e=P, R=0, work=None, nb=0, y=P, ydt=BF16, st=None))
    for K in (32, 512, 4096, 1 << 22):
        for m in range(5, 30):
            for n in range(0, 26):
                for M, N in ((1 << m, 1 << n), ((1 << m) - 15, max((1 << n) - 1, 1)), ((1 << m) - 1, 1 << n)):
                    if M * N > 1 << 34 or M * N * K <= 96e6:      # (small ones need no workspace and would run)
                        continue
                    assert dense(M=M, K=K, N=N) == INVALID and "workspace" in err(lib), (M, N, K)
                    for E in (1, 8000):
                        if M > E and M + 256 * E <= 1 << 29 and (M + 256 * E) * N <= 1 << 34:
                            assert gather(B=1, R=M, K=K, E=E, N=N) == INVALID and "workspace" in err(lib), (M, N, K, E)
    assert gather(B=1 << 20, R=1 << 20, K=4096, E=8, N=64) == UNSUPPORTED and "2^32 values" in err(lib)
    assert gather(B=1 << 27, R=1 << 27, K=32, E=8, N=64) == UNSUPPORTED and "2^32 values" in err(lib)
    assert gather(B=(1 << 20) - 1, R=(1 << 20) - 1, K=4096, E=8, N=64) == INVALID and "workspace" in err(lib)
    # what they said before: 2^26 columns and 2^35 outputs
    assert dense(M=(1 << 31) - 1, K=32, N=16) == UNSUPPORTED and "launch" in err(lib)
