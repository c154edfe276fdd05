"""Argument checks of rotary positions and of the 4-bit cache's entry points; no GPU: every rejection happens before
the device is touched."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "quantized_matmul_amd", "libqlin.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libqlin.so not built")

INVALID, UNSUPPORTED = 1, 2
F32, F16, BF16, U8 = 0, 1, 2, 3
P = 0x100000           # never dereferenced: validation rejects first
ODD = P + 1


@pytest.fixture(scope="module")
def lib():
    from quantized_matmul_amd import _binding
    return _binding.load_library()


def err(lib):
    return lib.qlin_last_error().decode()


def caller(f, base):
    return lambda **kw: f(*dict(base, **kw).values())


def cache(**kw):
    from quantized_matmul_amd._binding import _CacheStruct
    base = dict(k_codes=P, k_scales=P, k_biases=P, v_codes=P, v_scales=P, v_biases=P, mode=b"affine", pages=10, heads=4,
                page_size=16, head_dim=128, group_size=64, bits=4, dtype=BF16)
    base.update(kw)
    return ctypes.byref(_CacheStruct(*base.values()))


BAD_CACHES = [dict(mode=b"int4"), dict(mode=None), dict(group_size=16), dict(group_size=0), dict(mode=b"mxfp4"),
              dict(mode=b"nvfp4"), dict(dtype=U8), dict(pages=0), dict(heads=0), dict(page_size=0), dict(head_dim=0),
              dict(page_size=24), dict(page_size=8), dict(head_dim=96), dict(head_dim=48, group_size=32), dict(heads=-1)]
BIG_CACHES = [dict(mode=b"mxfp8"), dict(bits=8), dict(heads=4097), dict(head_dim=512), dict(page_size=1 << 25),
              dict(pages=1 << 28), dict(pages=(1 << 31) // 16, heads=1), dict(pages=1 << 26, heads=64)]
BAD_POINTERS = [dict(k_codes=None), dict(v_scales=None), dict(v_biases=None), dict(k_codes=P + 8), dict(k_scales=ODD),
                dict(v_biases=ODD), dict(mode=b"mxfp4", group_size=32), dict(v_codes=P + 4)]


@pytest.mark.parametrize("name", ["qlin_rotary", "qlin_rotary_grad"])
def test_rotary_rejects(lib, name):
    call = caller(getattr(lib, name), dict(x=P, dt=BF16, T=4, xs=256, heads=2, D=128, R=128, pos=P, freqs=P, inter=0,
                                           scale=1.0, y=P + (1 << 20), ys=256, st=None))
    for bad in (dict(dt=U8), dict(T=-1), dict(heads=0), dict(D=0), dict(D=100), dict(R=0), dict(R=3), dict(R=130),
                dict(scale=float("nan")), dict(scale=1e39), dict(xs=-1), dict(ys=255), dict(x=None), dict(y=None),
                dict(pos=None), dict(freqs=None), dict(x=ODD), dict(y=ODD), dict(pos=P + 2), dict(freqs=P + 2),
                dict(y=P + 2046), dict(y=P - 16), dict(y=P, ys=300), dict(xs=(1 << 31) + 1)):
        assert call(**bad) == INVALID, bad
        assert err(lib)
    assert call(D=264, R=8, ys=600) == UNSUPPORTED
    assert call(T=1 << 31) == UNSUPPORTED
    assert call(T=0, x=None, y=None, pos=None, freqs=None) == 0
    assert err(lib) == ""


def test_write_rejects(lib):
    call = caller(lib.qlin_kv_cache_write, dict(c=cache(), k=P, v=P, dt=BF16, T=3, ks=512, vs=512, slots=P, st=None))
    for kw in BAD_CACHES + BAD_POINTERS:
        assert call(c=cache(**kw)) == INVALID, kw
        assert err(lib)
    for kw in BIG_CACHES:
        assert call(c=cache(**kw)) == UNSUPPORTED, kw
    for bad in (dict(c=None), dict(dt=U8), dict(dt=F16), dict(T=-1), dict(ks=-1), dict(vs=(1 << 31) + 1), dict(k=None),
                dict(v=None), dict(slots=None), dict(k=ODD), dict(v=ODD), dict(slots=P + 2)):
        assert call(**bad) == INVALID, bad
    assert call(T=1 << 31) == UNSUPPORTED
    assert call(T=(1 << 27) + 1) == UNSUPPORTED and "2^36" in err(lib)
    assert call(T=0, k=None, v=None, slots=None, c=cache(k_codes=None)) == 0
    assert call(c=cache(mode=b"mxfp4", group_size=32, k_biases=None, v_biases=None, dtype=U8), dt=F32, T=0) == 0


def test_read_rejects(lib):
    call = caller(lib.qlin_kv_cache_read, dict(c=cache(), slots=P, T=3, k=P, v=P, dt=F32, st=None))
    for kw in BAD_CACHES + BAD_POINTERS:
        assert call(c=cache(**kw)) == INVALID, kw
    for kw in BIG_CACHES:
        assert call(c=cache(**kw)) == UNSUPPORTED, kw
    for bad in (dict(c=None), dict(dt=U8), dict(T=-1), dict(k=None), dict(v=None), dict(slots=None), dict(k=P + 8),
                dict(v=ODD), dict(slots=P + 2)):
        assert call(**bad) == INVALID, bad
    assert call(T=1 << 31) == UNSUPPORTED and call(T=(1 << 27) + 1) == UNSUPPORTED
    assert call(T=0, k=None, v=None, slots=None) == 0


def test_attention_rejects(lib):
    size = lib.qlin_kv_cache_attention_workspace_bytes
    need = size(cache(), BF16, 4, 16, 4, 300, 0, 0)
    assert need > 0
    base = dict(c=cache(), q=P, dt=BF16, T=4, qs=2048, qh=16, table=P, B=4, width=300, lengths=P, offsets=None, scale=0.1,
                causal=1, window=0, ws=P, nb=need, out=2 * P, st=None)
    call = caller(lib.qlin_kv_cache_attention, base)
    for kw in BAD_CACHES + BAD_POINTERS:
        assert call(c=cache(**kw)) == INVALID, kw
    for kw in BIG_CACHES:
        assert call(c=cache(**kw)) == UNSUPPORTED, kw
    for bad in (dict(c=None), dict(dt=U8), dict(dt=F16), dict(T=-1), dict(T=5), dict(qh=0), dict(qh=18), dict(B=3),
                dict(B=-1), dict(width=-1), dict(window=-1), dict(scale=float("inf")), dict(qs=-1), dict(qs=(1 << 31) + 1),
                dict(q=None), dict(table=None), dict(lengths=None), dict(out=None), dict(q=ODD), dict(out=P + 8),
                dict(table=P + 2), dict(lengths=P + 2), dict(offsets=P + 2), dict(ws=None), dict(nb=need - 1),
                dict(ws=P + 8), dict(out=P), dict(out=P + 3 * 4096 + 4080), dict(out=P - 4 * 4096 + 16)):
        assert call(**bad) == INVALID, bad
        assert err(lib)
    assert call(out=P) == INVALID and "overlaps" in err(lib)
    assert call(T=1 << 30, B=1 << 30) == UNSUPPORTED
    assert call(width=1 << 31) == UNSUPPORTED
    assert call(T=0, B=0, q=None, table=None, lengths=None, out=None, ws=None, nb=0) == 0
    assert size(cache(mode=b"x"), BF16, 4, 16, 4, 300, 0, 0) == 0
    assert size(cache(), BF16, 4, 16, 3, 300, 0, 0) == 0
    assert size(cache(dtype=F32), F32, 4, 16, 4, 300, 0, 0) == 0


def test_cache_struct_matches_the_header():
    """The header's fields, in order."""
    from quantized_matmul_amd._binding import _CacheStruct
    text = open(os.path.join(ROOT, "include", "qlin.h")).read()
    body = text[text.index("typedef struct qlin_kv_cache {") : text.index("} qlin_kv_cache;")]
    names = []
    for line in body.splitlines()[1:]:
        names += [w.strip().lstrip("*") for w in line.strip().rstrip(";").split(None, 1)[1].replace("char*", "").split(",")] \
            if line.strip() else []
    names = [n.split()[-1].lstrip("*") for n in names]
    assert names == [n for n, _ in _CacheStruct._fields_]
