"""Rows that a cache's write has to hold as qlin_quantize holds them, byte for byte, where its own arithmetic could
differ: groups of a few of the smallest fp32 steps, values that are no number."""
import numpy as np
import pytest
import torch

import oracle
from helpers import ORACLE_DT, to_oracle

pytestmark = pytest.mark.gpu

qm = pytest.importorskip("quantized_matmul_amd")

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FORMATS = [("affine", 32), ("affine", 64), ("affine", 128), ("mxfp4", 32), ("nvfp4", 16)]


def written(x, g, mode):
    """QuantizedWeight parts [rows, ...] of x [rows, D] from a cache's keys and from its values."""
    n, D = x.shape
    pages = -(-n // 16)
    cache = qm.kv_cache(pages, 1, 16, D, g, mode, x.dtype, DEV)
    slots = torch.arange(n, dtype=torch.int32, device=DEV)
    qm.kv_cache_write(cache, x[:, None].contiguous(), x[:, None].contiguous(), slots)
    return [[None if t is None else t.reshape(pages * 16, -1)[:n] for t in (w.value, w.scales, w.biases)]
            for w in (cache.key, cache.value)]


def same(a, b):
    """Equal bits; a NaN equals any NaN."""
    if a is None or not a.is_floating_point():
        return (a is None and b is None) or torch.equal(a, b)
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(7.0, 8.0, 9.0), b.nan_to_num(7.0, 8.0, 9.0))


@pytest.mark.parametrize("mode,g", FORMATS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_groups_of_the_smallest_numbers(dtype, mode, g):
    """Ranges of 1 to 300 of the type's smallest steps (a scale of few steps is far from range / 15), from zero, around
    it, and from some way off; and elements that are subnormal under a scale that is not."""
    D, least = 128, {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}[dtype]
    i = torch.arange(D, dtype=torch.float64)
    rows = []
    for span in list(range(1, 64)) + list(range(64, 300, 7)):
        rows += [(i * 5 % (span + 1)) * least, ((i * 3 % (span + 1)) - span // 2) * least, ((i % (span + 1)) + 1000) * least]
    for top in (1.0, 1.5, 2.0, 3.0, 6.0):                  # of a group, in quarters of the smallest normal number and below it
        for low in (1, 2, 3, 5, 7, 11):
            rows.append(torch.where(i % 16 == 3, top * 2.0 ** -124, (i % 8) * low * 2.0 ** -131))
    x = torch.stack(rows).to(DTYPES[dtype])
    want = oracle.quantize(to_oracle(x), ORACLE_DT[x.dtype], g, 4, mode)
    for side in written(x.to(DEV), g, mode):
        for t, w in zip(side, want):
            if t is not None:
                np.testing.assert_array_equal(to_oracle(t).reshape(w.shape), w)


@pytest.mark.parametrize("mode,g", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_values_that_are_no_number(dtype, mode, g):
    """NaN and infinities at every place of a group, alone and together: the bytes of `quantize`."""
    D = 128
    gen = torch.Generator().manual_seed(3)
    nan, inf = float("nan"), float("inf")
    rows = []
    for bad in ((nan,), (-nan,), (inf,), (-inf,), (nan, inf), (inf, nan), (-inf, inf), (nan, nan, -inf)):
        for at in list(range(0, 40)) + [63, 64, 72, 96, 120, 127]:
            x = torch.randn(D, generator=gen)
            for k, b in enumerate(bad):
                x[(at + 5 * k) % D] = b
            rows.append(x)
    rows += [torch.full((D,), nan), torch.full((D,), inf), torch.full((D,), -inf)]
    x = torch.stack(rows).to(DTYPES[dtype]).to(DEV)
    want = qm.quantize(x, g, 4, mode)
    for side in written(x, g, mode):
        for t, w in zip(side, (want.value, want.scales, want.biases)):
            assert same(t, w)
