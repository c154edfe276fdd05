"""Corners of the mixture-of-experts operators on the GPU against their 64-bit
statements (moe_reference)."""
import numpy as np
import pytest
import torch

import moe_reference as ref

pytestmark = pytest.mark.gpu

qm = pytest.importorskip("quantized_matmul_amd")

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def f64(t):
    return t.detach().cpu().double().numpy()


def full_route_grad(x, ids, g, score, scale):
    """Gradient of renormalized weights, every term of the chain rule kept: w_i = c s_i / S, S = sum s + 1e-20."""
    s, live = ref.scores(x, score), ids >= 0
    at = np.maximum(ids, 0)
    q, g = np.where(live, np.take_along_axis(s, at, 1), 0.0), np.where(live, g, 0.0)
    S = q.sum(1, keepdims=True) + 1e-20
    ds = scale * (g / S - (g * q).sum(1, keepdims=True) / S / S)
    full = np.zeros_like(s)
    for t in range(len(x)):
        full[t, ids[t][live[t]]] = ds[t][live[t]]
    if score == "sigmoid":
        return full * s * (1 - s)
    return s * (full - (full * s).sum(1, keepdims=True))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_gradient_of_scores_of_the_denominators_size(score, dtype):
    """A balance bias can choose experts whose scores sum to about the 1e-20 of the denominator. The weights then
    do move when all chosen logits move together, and through softmax with every other logit.

    Tolerances as for the route's gradient elsewhere: 1e-5 of the row's largest (terms of opposite sign cancel) and
    one rounding of the type; the formula against central differences of step 1e-5 with 1e-8 of the row's largest."""
    rng = np.random.default_rng(31)
    T, E, k, scale = 40, 30, 4, 2.5
    x = rng.normal(size=(T, E))
    x[:, 20:26] += (-42.5 if score == "softmax" else -46.0) + rng.uniform(-4, 4, (T, 1))
    x[3, 5] = -np.inf
    x = torch.from_numpy(x).to(DTYPES[dtype])
    b = torch.zeros(E)
    b[20:26] = 10.0
    g = torch.from_numpy(rng.normal(size=(T, k))).float()
    w, ids = qm.moe_route(x.to(DEV), k, score=score, bias=b.to(DEV), scale=scale)
    x64, g64 = f64(x), f64(g)
    rw, rids = ref.route(x64, k, score, bias=f64(b), scale=scale)
    np.testing.assert_array_equal(ids.cpu().numpy(), rids)
    np.testing.assert_allclose(f64(w), rw, rtol=4e-6)
    ids[::5, 2] = -1                                          # places left over
    rids[::5, 2] = -1
    r = full_route_grad(x64, rids, g64, score, scale)
    largest = np.abs(r).max(1, keepdims=True)
    if score == "softmax":                                    # the logits outside the choice take part
        assert (np.abs(r[:, :20]).max(1) / largest[:, 0]).max() > 0.1
    h, low = 1e-5, np.where(np.isfinite(x64), x64, -1e300)
    for e in range(E):
        d = np.zeros(E)
        d[e] = h
        slope = (ref.route_weights(low + d, rids, score, True, scale)
                 - ref.route_weights(low - d, rids, score, True, scale)) / (2 * h)
        np.testing.assert_array_less(np.abs((slope * g64).sum(1) - r[:, e]), 1e-8 * largest[:, 0] + 1e-12)
    got = f64(qm.moe_route_grad(x.to(DEV), ids, g.to(DEV), score=score, scale=scale))
    assert (np.abs(got - r) <= 1e-5 * largest + UNIT[dtype] * np.abs(r) + 1e-30).all(), np.abs(got - r).max()


def at_odd_address(scales, by):
    pad = torch.empty(scales.numel() + by, dtype=torch.uint8, device=DEV)
    pad[by:] = scales.reshape(-1)
    return pad[by:].view(scales.shape)


@pytest.mark.parametrize("by", [1, 4, 8])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("shape", [(300, 400, 1024), (5, 300, 512)])
def test_scales_at_odd_addresses_take_the_same_kernel(shape, codes, by):
    """Many rows by a weight whose scales are not 16-byte aligned: the path and the bits of aligned ones."""
    g = torch.Generator().manual_seed(41)
    N, K = shape[-2:]
    gather = shape[0] == 5
    w = torch.randn(shape if gather else (N, K), generator=g)
    qw = qm.quantize(w.to(DEV), mode="mxfp4")
    odd = qm.QuantizedWeight(qw.value, at_odd_address(qw.scales, by), None, 32, 4, True, "mxfp4")
    x = torch.randn((300, K), generator=g).bfloat16().to(DEV)
    ids = torch.randint(-1, 5, (300, 2), generator=g, dtype=torch.int32).to(DEV)
    xo = x
    if codes:
        x = qm.quantize(x, mode="mxfp4")
        xo = qm.QuantizedWeight(x.value, at_odd_address(x.scales, by), None, 32, 4, True, "mxfp4")
    run = (lambda a, b: qm.gather_mxfp4_matmul(a, b, ids)) if gather else qm.mxfp4_matmul
    y = run(x, qw)
    path = qm.last_path()
    assert path == ("mxfp4_gather_tiled" if gather else "mxfp4_tiled")
    for a, b in ((x, odd), (xo, odd), (xo, qw)):
        assert torch.equal(run(a, b), y)
        assert qm.last_path() == path
