"""Rotary positions and their gradient on the GPU against kv_reference in 64 bits.

Tolerance: the angle's turns are an fp64 product (2^-53 of them, nothing here), its fraction is rounded to fp32 once
(2^-24) and multiplied by 2 pi into at most pi / 4; sine and cosine are polynomials of about 4 roundings; two products
and a sum follow: together below 8 * 2^-24 of |a| + |b|, times scale; then one rounding of the type.
"""
import numpy as np
import pytest
import torch

import kv_reference as ref

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


def check(got, x, positions, freqs, dtype, **how):
    x64 = f64(x)
    want = ref.rotary(x64, positions.cpu().numpy(), freqs.cpu().numpy(), **how)
    size = np.abs(x64).max(-1, keepdims=True) * 2 * abs(how.get("scale", 1.0))
    tol = 8 * 2.0 ** -24 * size + UNIT[dtype] * np.abs(want) + (2.0 ** -25 if dtype == "f16" else 0)
    assert (np.abs(f64(got) - want) <= tol).all(), np.abs(f64(got) - want).max()


CASES = [
    # T, H, D, R, dtype, interleaved, scale
    (1, 40, 128, 128, "bf16", False, 1.0),
    (1, 1, 8, 2, "f32", True, 1.0),
    (3, 5, 64, 64, "f16", True, 1.0),
    (17, 3, 96, 64, "bf16", False, 0.5),
    (33, 7, 80, 80, "bf16", False, 1.0),      # half a row is no whole number of 16-byte runs in fp32 only
    (9, 2, 80, 22, "f16", False, 1.0),        # partners at odd places
    (9, 2, 72, 34, "f32", False, 1.3),
    (5, 4, 256, 256, "f32", False, 1.0),
    (5, 4, 256, 254, "f32", True, 1.0),
    (257, 2, 192, 96, "bf16", True, 1.0),
    (4100, 3, 64, 64, "bf16", False, 1.0),
    (70000, 1, 8, 8, "f16", False, 1.0),
]


@pytest.mark.parametrize("T,H,D,R,dtype,interleaved,scale", CASES)
def test_rotary_and_gradient(T, H, D, R, dtype, interleaved, scale):
    print(f"rotary T{T} H{H} D{D} R{R} {dtype} {'pairs' if interleaved else 'halves'}", flush=True)
    x = rand((T, H, D), dtype, T + D)
    pos = (torch.arange(T, dtype=torch.int32) * 13 % 100003 - 5).to(DEV)
    freqs = qm.rotary_frequencies(R, device=DEV)
    how = dict(interleaved=interleaved, scale=scale)
    check(qm.rotary(x, pos, freqs, **how), x, pos, freqs, dtype, **how)
    check(qm.rotary_grad(x, pos, freqs, **how), x, pos, freqs, dtype, backward=True, **how)


def test_gradient_is_the_slope():
    """Differences of rotary itself; it is linear, so they are exact up to the roundings of two outputs."""
    x, g = rand((2, 3, 16), "f32", 1), rand((2, 3, 16), "f32", 2)
    pos = torch.tensor([7, 100000], dtype=torch.int32, device=DEV)
    for interleaved in (False, True):
        freqs = qm.rotary_frequencies(12, device=DEV)
        grad = f64(qm.rotary_grad(g, pos, freqs, interleaved=interleaved, scale=1.5))
        for h in range(3):
            for d in range(16):
                step = torch.zeros_like(x)
                step[:, h, d] = 1.0
                slope = f64(qm.rotary(x + step, pos, freqs, interleaved=interleaved, scale=1.5)) \
                    - f64(qm.rotary(x - step, pos, freqs, interleaved=interleaved, scale=1.5))
                np.testing.assert_allclose((slope * f64(g)).sum((1, 2)) / 2, grad[:, h, d], atol=2e-5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_far_and_negative_positions(dtype):
    pos = torch.tensor([0, 1, -1, 1 << 20, (1 << 31) - 1, -(1 << 31), 65536, 99999], dtype=torch.int32, device=DEV)
    x = rand((8, 2, 32), dtype, 3)
    freqs = qm.rotary_frequencies(32, device=DEV)
    # 2^31 steps of angle 1: the turns hold 2^-53 * 2^31 / (2 pi) < 2^-24 turns, another 2 pi 2^-24 of the pair
    got, want = f64(qm.rotary(x, pos, freqs)), ref.rotary(f64(x), pos.cpu().numpy(), freqs.cpu().numpy())
    assert (np.abs(got - want) <= 16 * 2.0 ** -24 * 2 * np.abs(f64(x)).max() + UNIT[dtype] * np.abs(want)).all()


@pytest.mark.parametrize("R,interleaved", [(32, False), (32, True), (20, False), (10, False), (14, True)])
def test_strided_rows_and_in_place(R, interleaved):
    """Heads of a projection's row (odd offsets too), into rows of another stride, and over themselves."""
    freqs = qm.rotary_frequencies(R, device=DEV)
    pos = torch.arange(11, dtype=torch.int32, device=DEV) * 1000
    for lead in (0, 8, 3):
        row = rand((11, lead + 5 * 32 + 7), "bf16", lead + R)
        x = row[:, lead : lead + 160].view(11, 5, 32) if lead == 0 else row.as_strided((11, 5, 32), (row.shape[1], 32, 1), lead)
        plain = qm.rotary(x.contiguous(), pos, freqs, interleaved=interleaved)
        assert torch.equal(qm.rotary(x, pos, freqs, interleaved=interleaved), plain)
        wide = torch.full((11, 200), 9.0, dtype=torch.bfloat16, device=DEV)
        out = wide[:, :160].view(11, 5, 32) if False else wide.as_strided((11, 5, 32), (200, 32, 1), 0)
        qm.rotary(x, pos, freqs, interleaved=interleaved, out=out)
        assert torch.equal(out, plain) and (wide[:, 160:] == 9.0).all()
        before = row.clone()
        qm.rotary(x, pos, freqs, interleaved=interleaved, out=x)
        assert torch.equal(x, plain)
        row.as_strided((11, 5, 32), (row.shape[1], 32, 1), lead).copy_(before.as_strided((11, 5, 32), (row.shape[1], 32, 1), lead))
        assert torch.equal(row, before)      # nothing beside the heads was touched
    one = rand((1, 5, 32), "bf16", 9)
    same = one.expand(11, 5, 32)             # one row for all tokens
    assert torch.equal(qm.rotary(same, pos, freqs, interleaved=interleaved),
                       qm.rotary(same.contiguous(), pos, freqs, interleaved=interleaved))


def test_frequencies():
    base = 10000.0 ** -(np.arange(0, 64, 2) / 64)
    f = qm.rotary_frequencies(64, device="cpu").double().numpy()
    np.testing.assert_allclose(f, base, rtol=2 ** -24)
    np.testing.assert_allclose(qm.rotary_frequencies(64, factor=8.0, device="cpu").double().numpy(), base / 8, rtol=2 ** -24)
    b = qm.rotary_frequencies(64, factor=8.0, method="base", device="cpu").double().numpy()
    np.testing.assert_allclose(b[[0, -1]], [1.0, base[-1] / 8], rtol=2 ** -23)
    p = qm.rotary_frequencies(64, factor=8.0, method="parts", trained=4096, device="cpu").double().numpy()
    turns = 4096 * base / (2 * np.pi)
    np.testing.assert_allclose(p[turns >= 32], base[turns >= 32], rtol=2 ** -24)
    np.testing.assert_allclose(p[turns <= 1], base[turns <= 1] / 8, rtol=2 ** -24)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (p[mid] < base[mid]).all() and (p[mid] > base[mid] / 8).all()
    for bad in (dict(dim=3), dict(dim=0), dict(dim=8, factor=0.0), dict(dim=8, method="cubic"),
                dict(dim=2, method="base"), dict(dim=8, method="parts", slow=4.0, fast=4.0)):
        with pytest.raises(ValueError):
            qm.rotary_frequencies(**bad, device="cpu")


def test_refusals():
    x, pos, freqs = rand((4, 2, 32), "bf16", 1), torch.zeros(4, dtype=torch.int32, device=DEV), qm.rotary_frequencies(32, device=DEV)
    for bad in (lambda: qm.rotary(x.cpu(), pos, freqs), lambda: qm.rotary(x[0], pos, freqs),
                lambda: qm.rotary(x, pos[:3], freqs), lambda: qm.rotary(x, pos.long(), freqs),
                lambda: qm.rotary(x, pos, freqs.double()), lambda: qm.rotary(x.int(), pos, freqs),
                lambda: qm.rotary(x.transpose(1, 2), pos, freqs), lambda: qm.rotary(x, pos, freqs, out=x.float()),
                lambda: qm.rotary(x, pos, freqs, out=x[:3]), lambda: qm.rotary(x, pos.cpu(), freqs)):
        with pytest.raises(ValueError):
            bad()
    long = rand((5, 2, 32), "bf16", 2)
    for bad in (lambda: qm.rotary(x, pos, qm.rotary_frequencies(34, device=DEV)),
                lambda: qm.rotary(x, pos, freqs, scale=float("nan")),
                lambda: qm.rotary(long[:4], pos, freqs, out=long[1:]),              # overlaps x by three rows
                lambda: qm.rotary(x, pos, freqs, out=x.expand(1, 4, 2, 32)[0].as_strided((4, 2, 32), (0, 32, 1)))):
        with pytest.raises(qm.QlinError):
            bad()
    assert qm.rotary(x[:0], pos[:0], freqs).shape == (0, 2, 32)
