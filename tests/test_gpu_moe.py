"""Routing, mxfp4 products dense and by experts, and the weighted combine on
the GPU against their 64-bit statements (moe_reference).

Tolerances, from the arithmetic:
  router weights   fp32: exp and the quotients round within 4 ulp, a sum of E
                   positive terms within E/64 + 6 roundings of its order:
                   under 30 * 2^-24 for E <= 1024, taken as 4e-6 relative.
  router gradient  the same per term; terms of opposite sign cancel, so the
                   bound is absolute: 1e-5 of the row's largest, plus one
                   rounding of the output type.
  products         normwise 1e-5 sqrt(K) (fp32) or 2e-2 (16 bits), the
                   library's own for fp32 accumulation.
  combine          k + 2 roundings of 2^-24 of the terms' sizes, one of the type.
"""
import os

import numpy as np
import pytest
import torch

import moe_reference as ref
import synth
from helpers import normwise_rel_err, to_oracle, tolerance

pytestmark = pytest.mark.gpu

qm = pytest.importorskip("quantized_matmul_amd")

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def rand(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(DTYPES[dtype]).to(DEV)


def f64(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------ routing

ROUTES = [
    # T, E, k, dtype, score, bias, groups, kept, top, renorm, scale
    (1, 64, 8, "bf16", "softmax", False, 1, 1, 1, True, 1.0),
    (5, 60, 4, "f32", "softmax", False, 1, 1, 1, False, 1.0),
    (7, 1, 1, "f32", "sigmoid", False, 1, 1, 1, True, 1.0),
    (9, 3, 3, "f16", "softmax", True, 1, 1, 1, True, 2.5),
    (33, 128, 6, "f32", "sigmoid", True, 1, 1, 1, False, 1.0),
    (17, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True, 2.5),
    (13, 160, 6, "bf16", "softmax", False, 8, 3, 1, False, 16.0),
    (6, 100, 5, "f32", "sigmoid", True, 10, 2, 2, True, 1.0),
    (6, 72, 9, "f32", "softmax", True, 9, 5, 1, True, 1.0),
    (4, 300, 64, "f32", "softmax", False, 1, 1, 1, True, 1.0),
    (3, 1024, 16, "f32", "sigmoid", True, 64, 8, 2, True, 1.0),
    (3, 999, 8, "f16", "softmax", False, 1, 1, 1, False, 1.0),
    (70, 17, 17, "bf16", "sigmoid", False, 1, 1, 1, True, 1.0),
    (5, 128, 8, "f32", "sigmoid", True, 64, 20, 2, True, 1.0),
]


@pytest.mark.parametrize("T,E,k,dtype,score,bias,groups,kept,top,renorm,scale", ROUTES)
def test_route_and_gradient(T, E, k, dtype, score, bias, groups, kept, top, renorm, scale):
    print(f"route T{T} E{E} k{k} {dtype} {score} groups {groups}/{kept}/{top}", flush=True)
    x = rand((T, E), dtype, 100 + E, 1.5)
    b = rand((E,), "f32", 200 + E, 0.1) if bias else None
    how = dict(score=score, renormalize=renorm, scale=scale)
    w, ids = qm.moe_route(x, k, bias=b, groups=groups, groups_kept=kept, group_top=top, **how)
    rw, rids = ref.route(f64(x), k, bias=f64(b) if bias else None, groups=groups, groups_kept=kept, group_top=top,
                         **how)
    np.testing.assert_array_equal(ids.cpu().numpy(), rids)
    np.testing.assert_allclose(f64(w), rw, rtol=4e-6, atol=1e-30)
    g = rand((T, k), "f32", 300 + E)
    gx = qm.moe_route_grad(x, ids, g, **how)
    rg = ref.route_grad(f64(x), rids, f64(g), score, renorm, scale)
    tol = 1e-5 * np.abs(rg).max(1, keepdims=True) + UNIT[dtype] * np.abs(rg) + 1e-7
    assert (np.abs(f64(gx) - rg) <= tol).all(), np.abs(f64(gx) - rg).max()


def test_route_gradient_against_differences():
    x = rand((4, 40), "f32", 7)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            _, ids = qm.moe_route(x, 6, score=score, renormalize=renorm, scale=1.5)
            g = rand((4, 6), "f32", 8)
            got = f64(qm.moe_route_grad(x, ids, g, score=score, renormalize=renorm, scale=1.5))
            x64, i, h = f64(x), ids.cpu().numpy(), 1e-5
            for e in range(40):
                d = np.zeros_like(x64)
                d[:, e] = h
                slope = (ref.route_weights(x64 + d, i, score, renorm, 1.5)
                         - ref.route_weights(x64 - d, i, score, renorm, 1.5)) / (2 * h)
                np.testing.assert_allclose(got[:, e], (slope * f64(g)).sum(1), atol=2e-5 * np.abs(got).max() + 1e-7)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_gradient_where_it_vanishes(score):
    """Renormalized weights do not move with a single choice, nor under equal gradients: what is left is the
    1e-20 of the denominator, below 1e-14 here, where fp32 differences of weights would leave 1e-8."""
    x = rand((50, 20), "f32", 12, 2.0)
    for k, g in ((1, rand((50, 1), "f32", 13)), (5, torch.full((50, 5), 0.7, device=DEV))):
        _, ids = qm.moe_route(x, k, score=score, scale=2.5)
        assert qm.moe_route_grad(x, ids, g, score=score, scale=2.5).abs().max() <= 1e-14
    ids[:, 0], ids[::2, 3] = -1, -1                             # places left over, the first among them
    assert qm.moe_route_grad(x, ids, g, score=score, scale=2.5).abs().max() <= 1e-14
    if score == "sigmoid":                                      # scores of the denominator's size: it counts
        x = -46.0 + rand((50, 20), "f32", 14)
        _, ids = qm.moe_route(x, 4, score=score)
        g = rand((50, 4), "f32", 15)
        r = ref.route_grad(f64(x), ids.cpu().numpy(), f64(g), score, True, 1.0)
        np.testing.assert_allclose(f64(qm.moe_route_grad(x, ids, g, score=score)), r, rtol=1e-4,
                                   atol=1e-5 * np.abs(r).max())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_masks_and_empty_rows(score):
    inf = float("inf")
    low = torch.finfo(torch.float32).min
    x = torch.tensor([[1.0, 2.0, 2.0, -inf, float("nan"), 2.0, 0.0, 1.0],
                      [-inf] * 8,
                      [float("nan")] * 8,
                      [low] * 8,
                      [0.0] * 8,
                      [-inf, -inf, -inf, 5.0, -inf, -inf, -inf, -inf],
                      [inf, 1.0, -3.0, low, 80.0, 80.0, -90.0, 0.0]], device=DEV)
    w, ids = qm.moe_route(x, 6, score=score)
    rw, rids = ref.route(f64(x), 6, score)
    np.testing.assert_array_equal(ids.cpu().numpy(), rids)
    np.testing.assert_allclose(f64(w), rw, rtol=4e-6, atol=1e-30)
    assert (ids[1] == -1).all() and (w[1] == 0).all() and ids[5].tolist() == [3, -1, -1, -1, -1, -1]
    g = torch.ones_like(w)
    gx = qm.moe_route_grad(x, ids, g, score=score)
    assert torch.isfinite(gx).all() and (gx[1] == 0).all() and (gx[2] == 0).all() and gx[0, 3] == 0
    # a bias that is NaN or -inf takes its expert out, +inf puts it first
    b = torch.tensor([0.0, float("nan"), -inf, 0.0, 0.0, inf, 0.0, 0.0], device=DEV)
    _, ids = qm.moe_route(torch.zeros((1, 8), device=DEV), 8, score=score, bias=b)
    assert ids.tolist() == [[5, 0, 3, 4, 6, 7, -1, -1]]


def test_route_groups_without_experts():
    x = torch.full((2, 16), -float("inf"), device=DEV)
    x[0, 5] = 1.0                       # one free expert: three groups of four are empty
    w, ids = qm.moe_route(x, 4, groups=4, groups_kept=2, group_top=2, score="sigmoid")
    assert ids.tolist() == [[-1] * 4, [-1] * 4] or ids.tolist() == [[5, -1, -1, -1], [-1] * 4]
    rw, rids = ref.route(f64(x), 4, "sigmoid", groups=4, groups_kept=2, group_top=2)
    np.testing.assert_array_equal(ids.cpu().numpy(), rids)
    np.testing.assert_allclose(f64(w), rw, rtol=4e-6)


@pytest.mark.parametrize("E,groups", [(16, 4), (24, 8)])    # groups of whole lanes, and of others
def test_route_groups_with_infinite_biases(E, groups):
    per = E // groups
    x = rand((3, E), "f32", 11)
    x[1, 1:per] = -float("inf")         # the expert with the infinite bias is alone in its group
    b = torch.zeros(E, device=DEV)
    b[0] = float("inf")
    b[per] = -float("inf")
    for top in (1, 2):
        w, ids = qm.moe_route(x, 3, bias=b, groups=groups, groups_kept=2, group_top=top, score="sigmoid")
        rw, rids = ref.route(f64(x), 3, "sigmoid", bias=f64(b), groups=groups, groups_kept=2, group_top=top)
        np.testing.assert_array_equal(ids.cpu().numpy(), rids)
        np.testing.assert_allclose(f64(w), rw, rtol=4e-6)


def test_route_empty_and_shapes():
    w, ids = qm.moe_route(torch.empty((0, 8), device=DEV), 2)
    assert w.shape == (0, 2) and ids.dtype == torch.int32
    w, ids = qm.moe_route(rand((2, 3, 8), "bf16", 1), 2)
    assert w.shape == (2, 3, 2)
    with pytest.raises(ValueError):
        qm.moe_route(rand((4, 8), "f32", 1).t(), 2)
    with pytest.raises(ValueError):
        qm.moe_route(rand((4, 8), "f32", 1), 2, bias=torch.zeros(7, device=DEV))
    with pytest.raises(qm.QlinError):
        qm.moe_route(rand((4, 8), "f32", 1), 9)
    with pytest.raises(ValueError):
        qm.moe_route_grad(rand((4, 8), "f32", 1), ids, w)


# ----------------------------------------------------------------- products


def weight(shape, seed):
    w, _ = synth.normal(shape, 0.02, seed, synth.WEIGHT, "bf16")
    return qm.quantize(w.to(DEV), 32, 4, "mxfp4")


def values(qw):
    return ref.mxfp4_decode(to_oracle(qw.value), to_oracle(qw.scales))


def close(y, r, K):
    assert torch.isfinite(y).all()
    e = normwise_rel_err(y, r)
    assert e <= tolerance(y.dtype, K), e


@pytest.fixture(params=["chosen", "tiled"])
def form(request, monkeypatch):
    """Products by the kernel that their sizes choose, and by the tiled one."""
    if request.param == "tiled":
        monkeypatch.setenv("QLIN_MXFP4_TILE", "1")
    return request.param


def streams(R, N, K, E=None):
    """Whether a product chooses the streaming kernel; E: by experts."""
    if E is None:
        return R <= 16 or -(-R // 4) * N * K <= 24e6
    return R <= E or R * N * K <= 48e6


DENSE = [(1, 16, 32), (1, 1, 64), (2, 17, 96), (3, 130, 160), (15, 48, 512), (16, 33, 544), (17, 64, 480),
         (31, 257, 1024), (33, 100, 2080), (64, 128, 256), (65, 128, 256), (65, 31, 32), (100, 130, 96),
         (129, 257, 544), (300, 300, 1056), (257, 129, 1536), (512, 256, 4096)]


@pytest.mark.parametrize("M,N,K", DENSE)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_dense_product(M, N, K, dtype, form):
    print(f"mxfp4_matmul M{M} N{N} K{K} {dtype} {form}", flush=True)
    qw, x = weight((N, K), 400 + N), rand((M, K), dtype, 500 + M)
    y = qm.mxfp4_matmul(x, qw)
    assert y.dtype == x.dtype and qm.last_path() == ("mxfp4_stream" if form == "chosen" and streams(M, N, K) else "mxfp4_tiled")
    close(y, ref.mxfp4_round(f64(x)) @ values(qw).T, K)
    # the same codes given as such: the same bits
    if dtype != "f16":
        qx = qm.quantize(x, 32, 4, "mxfp4")
        y2 = qm.mxfp4_matmul(qx, qw, out_dtype=x.dtype)
        assert torch.equal(y2, y)


@pytest.mark.parametrize("M,N,K", [(1, 64, 96), (40, 130, 544), (200, 257, 320)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_dense_product_swiglu(M, N, K, dtype, form):
    qw, x = weight((N, K), 410 + N), rand((M, 2 * K), dtype, 510 + M)
    y = qm.mxfp4_matmul(x, qw, activation="swiglu")
    close(y, ref.mxfp4_round(ref.swiglu(f64(x))) @ values(qw).T, K)


@pytest.mark.parametrize("M", [3, 80])
def test_dense_product_types_and_unaligned_views(M, form):
    N, K = 70, 288
    qw = weight((N, K), 420)
    flat = rand((M * K + 1,), "bf16", 520)
    x = flat[1:].view(M, K)                                     # 2-byte aligned
    r = ref.mxfp4_round(f64(x)) @ values(qw).T
    for dt in (torch.float32, torch.float16, torch.bfloat16):
        close(qm.mxfp4_matmul(x, qw, out_dtype=dt), r, K)
    pad = torch.empty(qw.scales.numel() + 3, dtype=torch.uint8, device=DEV)
    pad[3:] = qw.scales.reshape(-1)
    odd = qm.QuantizedWeight(qw.value, pad[3:].view(qw.scales.shape), None, 32, 4, True, "mxfp4")
    assert torch.equal(qm.mxfp4_matmul(x, odd), qm.mxfp4_matmul(x, qw))


@pytest.mark.parametrize("M", [5, 150])
def test_dense_product_long_scale_rows_at_odd_addresses(M, form):
    """K a multiple of 512 with scales that are not 16-byte aligned."""
    N, K = 130, 1024
    qw, x = weight((N, K), 421), rand((M, K), "bf16", 521)
    pad = torch.empty(qw.scales.numel() + 5, dtype=torch.uint8, device=DEV)
    pad[5:] = qw.scales.reshape(-1)
    odd = qm.QuantizedWeight(qw.value, pad[5:].view(qw.scales.shape), None, 32, 4, True, "mxfp4")
    r = ref.mxfp4_round(f64(x)) @ values(qw).T
    close(qm.mxfp4_matmul(x, odd), r, K)
    qx = qm.quantize(x, 32, 4, "mxfp4")
    xpad = torch.empty(qx.scales.numel() + 1, dtype=torch.uint8, device=DEV)
    xpad[1:] = qx.scales.reshape(-1)
    qx.scales = xpad[1:].view(qx.scales.shape)
    close(qm.mxfp4_matmul(qx, odd), r, K)


@pytest.mark.parametrize("M", [4, 90])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_dense_product_marks_blocks_that_are_not_finite(M, bad, form):
    qw, x = weight((40, 128), 430), rand((M, 128), "bf16", 530)
    clean = qm.mxfp4_matmul(x, qw)
    x[1, 77] = bad
    y = qm.mxfp4_matmul(x, qw)
    assert torch.isnan(y[1]).all()
    keep = torch.arange(M, device=DEV) != 1
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("M", [2, 12, 40])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_activation_rounding_is_exact(M, dtype, form):
    """Against the identity the product gives the rounded activation itself:
    E2M1 ties and their neighbours at many scales, tiny blocks, signed zeros."""
    K = 160
    rng = np.random.default_rng(77)
    ties = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7])
    top = {"bf16": 60, "f16": 8, "f32": 60}[dtype]
    v = rng.choice(ties, (M, K // 32, 32)) * (1 + rng.integers(-1, 2, (M, K // 32, 32)) * UNIT[dtype] * 2)
    v *= rng.choice([-1.0, 1.0], v.shape) * np.exp2(rng.integers(-top, top, (M, K // 32, 1)))
    v[0, 0] = 0.0
    v[1, 1] = -0.0
    v[1, 2] *= {"bf16": 1e-30, "f16": 1e-3, "f32": 1e-36}[dtype]        # down to the type's subnormals
    x = torch.from_numpy(v.reshape(M, K)).to(DTYPES[dtype]).to(DEV)
    eye = qm.quantize(torch.eye(K, device=DEV), 32, 4, "mxfp4")
    assert np.array_equal(values(eye), np.eye(K))
    y = qm.mxfp4_matmul(x, eye, out_dtype=torch.float32)
    np.testing.assert_array_equal(f64(y), ref.mxfp4_round(f64(x)))


@pytest.mark.parametrize("scale", [1e-30, 1e30, 0.0])
def test_dense_product_extreme_values(scale, form):
    qw = weight((32, 64), 440)
    x = rand((3, 64), "f32", 540) * scale
    x[0, 32:] = 0.0
    y = qm.mxfp4_matmul(x, qw)
    r = ref.mxfp4_round(f64(x)) @ values(qw).T
    assert normwise_rel_err(y, r) <= tolerance(torch.float32, 64)


def choices(B, k, E, seed, dropped=0.0, one=None):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] if k <= E else rng.integers(0, E, k) for _ in range(B)]).astype(np.int32)
    ids[rng.random(ids.shape) < dropped] = -1
    if one is not None:
        ids[:] = one
    return ids


GATHER = [
    # B, k, E, N, K, dropped, one expert
    (1, 8, 64, 48, 96, 0.0, None),
    (2, 4, 16, 33, 544, 0.3, None),
    (1, 1, 1, 20, 32, 0.0, None),
    (5, 3, 4, 130, 160, 0.1, None),
    (40, 2, 4, 64, 512, 0.0, None),
    (60, 2, 3, 65, 480, 0.2, None),
    (50, 4, 8, 70, 256, 0.0, 5),
    (30, 2, 8, 70, 256, 0.0, -1),
    (200, 2, 5, 140, 96, 0.1, None),
    (300, 4, 6, 129, 1056, 0.05, None),
    (300, 1, 3, 300, 512, 0.0, 2),
    (150, 2, 3, 40, 64, 0.0, -1),
    (2600, 2, 7, 64, 128, 0.02, None),
    (100, 2, 3, 1040, 1056, 0.1, None),
    (1700, 4, 9, 40, 64, 0.02, None),
    (3000, 3, 300, 33, 96, 0.0, None),
]


@pytest.mark.parametrize("B,k,E,N,K,dropped,one", GATHER)
def test_gather_product(B, k, E, N, K, dropped, one, form):
    print(f"gather_mxfp4_matmul B{B} k{k} E{E} N{N} K{K} {form}", flush=True)
    qw, x = weight((E, N, K), 600 + N), rand((B, K), "bf16", 700 + B)
    ids = choices(B, k, E, 800 + B, dropped, one)
    t = torch.from_numpy(ids).to(DEV)
    y = qm.gather_mxfp4_matmul(x, qw, t, out_dtype=torch.float32)
    stream = form == "chosen" and streams(B * k, N, K, E)
    assert qm.last_path() == ("mxfp4_gather_stream" if stream else "mxfp4_gather_tiled") and y.shape == (B, k, N)
    r = ref.gather_product(ref.mxfp4_round(f64(x)), values(qw), ids)
    close(y, r, K)
    assert (y[t < 0] == 0).all()
    qx = qm.quantize(x, 32, 4, "mxfp4")
    assert torch.equal(qm.gather_mxfp4_matmul(qx, qw, t, out_dtype=torch.float32), y)


@pytest.mark.parametrize("B,E", [(3, 32), (90, 8), (700, 4)])
def test_gather_product_swiglu_and_types(B, E, form):
    N, K = 72, 224
    qw, x = weight((E, N, K), 610), rand((B, 2 * K), "f16", 710)
    ids = choices(B, 1, E, 810, 0.1)
    t = torch.from_numpy(ids).to(DEV)
    y = qm.gather_mxfp4_matmul(x, qw, t, activation="swiglu")
    r = ref.gather_product(ref.mxfp4_round(ref.swiglu(f64(x))), values(qw), ids)
    close(y, r, K)
    y1 = qm.gather_mxfp4_matmul(x, qw, t[:, 0].contiguous(), activation="swiglu")
    assert y1.shape == (B, N) and torch.equal(y1, y[:, 0])


def test_gather_product_experts_out_of_range(form):
    qw, x = weight((4, 32, 64), 620), rand((100, 64), "bf16", 720)
    ids = choices(100, 2, 4, 820)
    ids[::3, 1] = 4
    ids[5, 0] = np.iinfo(np.int32).max
    ids[6, 0] = np.iinfo(np.int32).min
    y = qm.gather_mxfp4_matmul(x, qw, torch.from_numpy(ids).to(DEV))
    bad = (ids < 0) | (ids >= 4)
    assert (f64(y)[bad] == 0).all()
    close(y, ref.gather_product(ref.mxfp4_round(f64(x)), values(qw), ids), 64)


def test_gather_product_many_rows():
    """More chunks of rows than each scans for itself: the same bits as in parts."""
    qw, x = weight((5, 20, 64), 622), rand((160000, 64), "bf16", 722)
    ids = torch.randint(-1, 6, (160000, 2), dtype=torch.int32, device=DEV)
    y = qm.gather_mxfp4_matmul(x, qw, ids)
    assert qm.last_path() == "mxfp4_gather_tiled"
    for m in range(0, 160000, 80000):
        assert torch.equal(y[m:m + 80000], qm.gather_mxfp4_matmul(x[m:m + 80000], qw, ids[m:m + 80000])), m


def test_gather_product_many_experts(form):
    E = 3000
    qw, x = weight((E, 16, 32), 621), rand((2000, 32), "bf16", 721)
    ids = choices(2000, 3, E, 821, 0.01)
    y = qm.gather_mxfp4_matmul(x, qw, torch.from_numpy(ids).to(DEV), out_dtype=torch.float32)
    close(y, ref.gather_product(ref.mxfp4_round(f64(x)), values(qw), ids), 32)


def test_products_refuse(monkeypatch):
    qw, x = weight((32, 64), 630), rand((4, 64), "bf16", 730)
    ids = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    q8 = qm.quantize(rand((32, 64), "bf16", 1), 32, 8, "mxfp8")
    for f in (lambda: qm.mxfp4_matmul(x, q8), lambda: qm.mxfp4_matmul(rand((4, 96), "bf16", 2), qw),
              lambda: qm.mxfp4_matmul(x, qw, activation="swiglu"), lambda: qm.mxfp4_matmul(x.t(), qw),
              lambda: qm.gather_mxfp4_matmul(x, qw, ids), lambda: qm.mxfp4_matmul(x.int(), qw),
              lambda: qm.mxfp4_matmul(x.cpu(), qw), lambda: qm.mxfp4_matmul(q8, qw)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(qm.QlinError):
        qm.mxfp4_matmul(x, qw, activation="tanh")
    monkeypatch.setenv("QLIN_MXFP4_TILE", "1")
    with pytest.raises(qm.QlinError):
        qm.mxfp4_matmul(x.repeat(10, 1), qw, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    qe = weight((2, 32, 64), 631)
    for bad in (ids.long(), ids[:3], ids[:, :1].expand(4, 2)):
        with pytest.raises(ValueError):
            qm.gather_mxfp4_matmul(x, qe, bad)
    assert qm.mxfp4_matmul(x[:0], qw).shape == (0, 32)
    assert qm.gather_mxfp4_matmul(x[:0], qe, ids[:0]).shape == (0, 2, 32)
    assert qm.gather_mxfp4_matmul(x, qe, ids[:, :0]).shape == (4, 0, 32)


@pytest.mark.parametrize("tile", ["0", "1", "2", "3", "4"])
@pytest.mark.parametrize("M,N,K", [(17, 70, 96), (130, 300, 544), (300, 513, 1056)])
def test_every_tile(M, N, K, tile, monkeypatch):
    """Each shape of the tiled kernel's workgroup, dense and by experts, in every output type."""
    monkeypatch.setenv("QLIN_MXFP4_TILE", tile)
    qw, x = weight((3, N, K), 650 + N), rand((M, K), "bf16", 750 + M)
    ids = choices(M, 2, 3, 850, 0.1)
    t, w, x64 = torch.from_numpy(ids).to(DEV), values(qw), ref.mxfp4_round(f64(x))
    first = qm.QuantizedWeight(qw.value[0], qw.scales[0], None, 32, 4, True, "mxfp4")
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        print(f"tile {tile} M{M} N{N} K{K} {dt}", flush=True)
        close(qm.mxfp4_matmul(x, first, out_dtype=dt), x64 @ w[0].T, K)
        assert qm.last_path() == "mxfp4_tiled"
        close(qm.gather_mxfp4_matmul(x, qw, t, out_dtype=dt), ref.gather_product(x64, w, ids), K)
        assert qm.last_path() == "mxfp4_gather_tiled"


@pytest.mark.parametrize("tile", ["0", "1", "2", "3", "4"])
@pytest.mark.parametrize("M", [70, 300])
def test_tiled_product_reads_no_stale_lds(M, tile, monkeypatch):
    """With the whole LDS filled with NaN before each tile the output is the same."""
    monkeypatch.setenv("QLIN_MXFP4_TILE", tile)
    qw, x = weight((200, 1056), 640), rand((M, 1056), "bf16", 740)
    y = qm.mxfp4_matmul(x, qw)
    qe, ids = weight((2, 200, 1056), 641), torch.from_numpy(choices(M, 1, 2, 841)).to(DEV)
    ye = qm.gather_mxfp4_matmul(x, qe, ids)
    monkeypatch.setenv("QLIN_DEBUG_LDS_NAN", "1")
    assert torch.equal(qm.mxfp4_matmul(x, qw), y)
    assert torch.equal(qm.gather_mxfp4_matmul(x, qe, ids), ye)


# ------------------------------------------------------------------ combine

COMBINE = [(1, 1, 1), (1, 8, 64), (3, 2, 7), (5, 3, 8), (2, 4, 2056), (33, 6, 515), (17, 8, 1024), (4, 64, 24),
           (260, 2, 96)]


@pytest.mark.parametrize("T,k,D", COMBINE)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dropped", [False, True])
def test_combine_and_gradient(T, k, D, dtype, dropped):
    h, w, gy = rand((T, k, D), dtype, 900 + D), rand((T, k), "f32", 901), rand((T, D), dtype, 902)
    ids = None
    if dropped:
        ids = choices(T, k, max(k, 4), 903, 0.4)
        ids[0] = -1
        h[torch.from_numpy(ids < 0).to(DEV)] = float("nan")        # never read
    n = None if ids is None else ids
    t = None if ids is None else torch.from_numpy(ids).to(DEV)
    h64, w64, g64 = f64(h), f64(w), f64(gy)
    y = f64(qm.moe_combine(h, w, t))
    r = ref.combine(h64, w64, n)
    size = ref.combine(np.abs(h64), np.abs(w64), n)
    assert (np.abs(y - r) <= (k + 2) * 2.0 ** -24 * size + UNIT[dtype] * np.abs(r) + 1e-7 * (dtype == "f16")).all()
    gh, gw = qm.moe_combine_grad(gy, h, w, t)
    rh, rw = ref.combine_grad(g64, h64, w64, n)
    assert (np.abs(f64(gh) - rh) <= (UNIT[dtype] + 2.0 ** -23) * np.abs(rh) + 1e-7 * (dtype == "f16")).all()
    total = ref.combine_grad(np.abs(g64), np.abs(h64), w64, n)[1]
    assert (np.abs(f64(gw) - rw) <= (D / 64 + 16) * 2.0 ** -24 * total).all()


def test_combine_unaligned_views_and_refusals():
    flat = rand((3 * 2 * 16 + 1,), "bf16", 910)
    h, w = flat[1:].view(3, 2, 16), rand((3, 2), "f32", 911)
    np.testing.assert_allclose(f64(qm.moe_combine(h, w)), ref.combine(f64(h), f64(w)), atol=2.0 ** -6)
    assert qm.moe_combine(h[:0], w[:0]).shape == (0, 16)
    gh, gw = qm.moe_combine_grad(h[:0, 0], h[:0], w[:0])
    assert gh.shape == (0, 2, 16) and gw.shape == (0, 2)
    for f in (lambda: qm.moe_combine(h, w.half()), lambda: qm.moe_combine(h, w[:2]),
              lambda: qm.moe_combine(h, w, torch.zeros((3, 2), dtype=torch.int64, device=DEV)),
              lambda: qm.moe_combine_grad(w, h, w)):
        with pytest.raises(ValueError):
            f()


# ------------------------------------------------------- streams and graphs


def layer(x, logits, up, down, k):
    w, ids = qm.moe_route(logits, k)
    h = qm.gather_mxfp4_matmul(x, up, ids)
    B, _, D = h.shape
    o = qm.gather_mxfp4_matmul(h.view(B * k, D), down, ids.view(B * k), activation="swiglu")
    return qm.moe_combine(o.view(B, k, -1), w, ids)


@pytest.mark.parametrize("B", [2, 40, 600])
def test_layer_on_another_stream_and_in_a_graph(B):
    E, k, D, F = 8, 2, 128, 96
    up, down = weight((E, 2 * F, D), 950), weight((E, D, F), 951)
    x, logits = rand((B, D), "bf16", 952), rand((B, E), "f32", 953)
    y = layer(x, logits, up, down, k)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x2 = x * 1.0                                  # made on the side stream: nothing else orders it
        y2 = layer(x2, logits, up, down, k)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y2, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer(x, logits, up, down, k)
    for rep in range(3):
        out.zero_()
        (x.float() * 2).sum()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y), rep


# ------------------------------------------------- more than one launch holds

def enough(gigabytes):
    free = torch.cuda.mem_get_info()[0]
    if free < gigabytes * 10 ** 9:
        pytest.skip(f"needs {gigabytes} GB of device memory")


def test_route_of_more_tokens_than_a_launch_holds():
    enough(12)
    T, E = 2 ** 28 + 5, 3                                    # 16 lanes a token
    x = torch.empty((T, E), dtype=torch.bfloat16, device=DEV).normal_()
    w, ids = qm.moe_route(x, 1)
    for t in range(0, T, 2 ** 26):
        pw, pids = qm.moe_route(x[t:t + 2 ** 26], 1)
        assert torch.equal(w[t:t + 2 ** 26], pw) and torch.equal(ids[t:t + 2 ** 26], pids), t
    T = 2 ** 26 + 5                                          # a wave a token
    x, ids = x[:T], ids[:T]
    g = torch.empty((T, 1), device=DEV).normal_()
    gx = qm.moe_route_grad(x, ids, g, renormalize=False)
    for t in range(0, T, 2 ** 24):
        s = slice(t, t + 2 ** 24)
        assert torch.equal(gx[s], qm.moe_route_grad(x[s], ids[s], g[s], renormalize=False)), t


def test_combine_of_more_values_than_a_launch_holds():
    enough(40)
    T, D = 3, 2 ** 31 - 1                                    # a thread a value
    h = torch.empty((T, 1, D), dtype=torch.bfloat16, device=DEV).normal_()
    w = torch.tensor([[0.5], [1.25], [-3.0]], device=DEV)
    y = qm.moe_combine(h, w)
    for t in range(T):
        for d in range(0, D, 2 ** 28):
            s = slice(d, d + 2 ** 28)
            assert torch.equal(y[t, s], (w[t] * h[t, 0, s].float()).bfloat16()), (t, d)
    del h, y
    T, D = 2 ** 26 + 3, 8                                    # a wave a row
    h = torch.empty((T, 1, D), dtype=torch.bfloat16, device=DEV).normal_()
    gy = torch.empty((T, D), dtype=torch.bfloat16, device=DEV).normal_()
    w = torch.empty((T, 1), device=DEV).normal_()
    gh, gw = qm.moe_combine_grad(gy, h, w)
    for t in range(0, T, 2 ** 24):
        s = slice(t, t + 2 ** 24)
        assert torch.equal(gh[s, 0], (w[s] * gy[s].float()).bfloat16()), t
        terms = gy[s].double() * h[s, 0].double()
        assert ((gw[s, 0] - terms.sum(1)).abs() <= 8 * 2.0 ** -24 * terms.abs().sum(1)).all(), t


def test_product_of_more_words_than_a_launch_holds():
    enough(100)
    M, N, K = 2 ** 22 + 1, 16, 8192                          # a thread a word of x; small integers: sums are exact
    x = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    for m in range(0, M, 2 ** 18):
        x[m:m + 2 ** 18].random_(-6, 7)
    qw = qm.quantize(torch.empty((N, K), dtype=torch.bfloat16, device=DEV).random_(-6, 7), mode="mxfp4")
    y = qm.mxfp4_matmul(x, qw, out_dtype=torch.float32)
    for m in range(0, M, 2 ** 20):
        assert torch.equal(y[m:m + 2 ** 20], qm.mxfp4_matmul(x[m:m + 2 ** 20], qw, out_dtype=torch.float32)), m


def test_large_calls_that_pass_the_caches():
    """Calls of over 192 MB store (and read x) with other instructions: the same bits as in parts."""
    qw = weight((6200, 96), 980)
    x = torch.empty((8192, 96), dtype=torch.bfloat16, device=DEV).normal_()
    y = qm.mxfp4_matmul(x, qw, out_dtype=torch.float32)
    qe = weight((4, 6200, 96), 981)
    ids = torch.randint(-1, 4, (8192, 1), dtype=torch.int32, device=DEV)
    ye = qm.gather_mxfp4_matmul(x, qe, ids, out_dtype=torch.float32)
    for m in range(0, 8192, 1024):
        s = slice(m, m + 1024)
        assert torch.equal(y[s], qm.mxfp4_matmul(x[s], qw, out_dtype=torch.float32)), m
        assert torch.equal(ye[s], qm.gather_mxfp4_matmul(x[s], qe, ids[s], out_dtype=torch.float32)), m
    qw = weight((40, 4096), 982)
    x = torch.empty((16000, 8192), dtype=torch.float16, device=DEV).normal_()
    y = qm.mxfp4_matmul(x, qw, activation="swiglu")
    for m in range(0, 16000, 1000):
        assert torch.equal(y[m:m + 1000], qm.mxfp4_matmul(x[m:m + 1000], qw, activation="swiglu")), m
    h, w = torch.empty((6000, 3, 4096), dtype=torch.bfloat16, device=DEV).normal_(), torch.rand((6000, 3), device=DEV)
    gy = torch.empty((6000, 4096), dtype=torch.bfloat16, device=DEV).normal_()
    y, (gh, gw) = qm.moe_combine(h, w), qm.moe_combine_grad(gy, h, w)
    for t in range(0, 6000, 1000):
        s = slice(t, t + 1000)
        assert torch.equal(y[s], qm.moe_combine(h[s], w[s])), t
        pgh, pgw = qm.moe_combine_grad(gy[s], h[s], w[s])
        assert torch.equal(gh[s], pgh) and torch.equal(gw[s], pgw), t
