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


def near_ties(dtype, M, K, seed):
    """x [M, 2 K] whose silu(gate) * up lies near ties of its block's 4-bit codes; gates from -80 to 20."""
    rng = np.random.default_rng(seed)
    gate = torch.from_numpy(rng.uniform(-80, 20, (M, K // 32, 1)) + rng.uniform(-3, 3, (M, K // 32, 32))).to(DTYPES[dtype])
    g = f64(gate)
    tie = rng.choice([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0], g.shape)
    tie[:, :, 0] = 4.7                                        # the block's largest magnitude or next to it
    want = tie * (1 + rng.uniform(-2.0 ** -17, 2.0 ** -17, g.shape)) * rng.choice([-1.0, 1.0], g.shape)
    up = want / (g / (1 + np.exp(-g)))
    up = up / np.exp2(np.rint(np.log2(np.abs(up[:, :, :1]))))  # the first value's up near 1
    if dtype == "f16":
        up = np.clip(up, -60000, 60000)
    x = torch.cat([gate.reshape(M, K), torch.from_numpy(up).reshape(M, K).to(DTYPES[dtype])], 1)
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_swiglu_rounds_to_codes_within_its_stated_error(dtype):
    """silu(gate) * up carries a relative error of at most d = (1.25 |gate| + 7) 2^-24: the argument of 2^x is rounded
    (2^-24 of itself, and log2 e is within 2^-26), then come 2^x and 1 / x (2^-23 each) and three roundings. So each
    code lies between those of v (1 - d) and v (1 + d), which are equal but next to a tie."""
    M, K = 64, 160
    x = near_ties(dtype, M, K, 61)
    g, v = f64(x)[:, :K], ref.swiglu(f64(x))
    d = (1.25 * np.abs(g) + 7) * 2.0 ** -24
    a, b = ref.mxfp4_round(v * (1 - d)), ref.mxfp4_round(v * (1 + d))
    top = [np.floor(np.log2(np.abs(v * f).reshape(M, -1, 32).max(2))) for f in (1 - d, 1 + d)]
    assert (top[0] == top[1]).all()                           # no block's exponent hangs on the error
    eye = qm.quantize(torch.eye(K, device=DEV), mode="mxfp4")
    y = f64(qm.mxfp4_matmul(x.to(DEV), eye, activation="swiglu", out_dtype=torch.float32))
    assert ((np.minimum(a, b) <= y) & (y <= np.maximum(a, b))).all()
    if dtype == "f32":
        assert (a != b).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_activation_rounding_of_the_smallest_blocks(dtype):
    """Blocks whose largest value is about the type's least normal number and below, ties and their neighbours among
    the values: exact, as against an identity of 2^40 whose products are normal numbers."""
    M, K = 48, 160
    rng = np.random.default_rng(51)
    ties = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7])
    v = rng.choice(ties, (M, K // 32, 32)) * (1 + rng.integers(-1, 2, (M, K // 32, 32)) * UNIT[dtype] * 2)
    low, high = (-24, -10) if dtype == "f16" else (-135, -118)
    v *= rng.choice([-1.0, 1.0], v.shape) * np.exp2(rng.integers(low, high, (M, K // 32, 1)))
    x = torch.from_numpy(v.reshape(M, K)).to(DTYPES[dtype])
    eye = qm.quantize(torch.eye(K, device=DEV) * 2.0 ** 40, mode="mxfp4")
    y = qm.mxfp4_matmul(x.to(DEV), eye, out_dtype=torch.float32)
    np.testing.assert_array_equal(f64(y), ref.mxfp4_round(f64(x)) * 2.0 ** 40)
