"""Attention over a 4-bit cache on the GPU: what the matrix cores' 16-bit operands may cost. Problems and formulas are those
of test_gpu_kv_attention, tolerances narrower where a rounding is left out."""
import pytest
import torch

from test_gpu_kv_attention import DEV, DTYPES, Problem, rand

pytestmark = pytest.mark.gpu

qm = pytest.importorskip("quantized_matmul_amd")


@pytest.mark.parametrize("rows", [1, 5, 40, 300])
@pytest.mark.parametrize("dtype,mode,g", [("bf16", "mxfp4", 32), ("f16", "mxfp4", 32), ("bf16", "nvfp4", 16), ("f16", "nvfp4", 16),
                                          ("f16", "affine", 32), ("f16", "affine", 128)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_equal_values_come_out_as_they_are(D, dtype, mode, g, rows):
    """Weights of a row add up to one as they multiply the values: where all keys have the same values (and those, rounded
    once, are numbers of the type), so has the output, to the bit."""
    if D % g:
        pytest.skip("head_dim is no multiple of the group")
    print(f"equal values D{D} {dtype} {mode} g{g} rows {rows}", flush=True)
    window = 6                                               # few keys: what is lost does not average out
    p = Problem([rows] * 3, [rows + 3, rows + 40, max(rows, 2)], 2, 3, D, mode, g, dtype, 16, seed=46, garbage=False)
    one = rand((1, 2, 1, D), dtype, 47)
    w = qm.quantize(one.expand(p.cache.pages, 2, 16, D).contiguous(), g, 4, mode)
    p.cache = qm.KVCache(p.cache.key, w)
    got = p.call(window=window)
    want = torch.from_numpy(p.dense()[1][0, :, 0]).to(DTYPES[dtype]).to(DEV).repeat_interleave(3, 0)
    assert torch.equal(got, want.expand_as(got))
