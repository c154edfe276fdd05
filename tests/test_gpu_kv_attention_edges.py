"""Attention over a 4-bit cache on the GPU where blocks of keys hold no values. Problems, formulas and tolerances are those of test_gpu_kv_attention."""
import pytest
import torch

from test_gpu_kv_attention import DEV, Problem

pytestmark = pytest.mark.gpu

qm = pytest.importorskip("quantized_matmul_amd")


@pytest.mark.parametrize("size", [1.0, 1e-5, 1e-30])
@pytest.mark.parametrize("mode,g", [("affine", 64), ("affine", 32), ("mxfp4", 32)])
@pytest.mark.parametrize("rows", [1, 90, 300])
def test_blocks_without_values_beside_small_ones(rows, mode, g, size):
    """A page of zeros and pages that are not there, before, among and behind values of any size, and a sequence whose
    values are all zero: the others keep their bits, whose tolerance is relative to them alone."""
    print(f"empty blocks rows {rows} {mode} g{g} size {size}", flush=True)
    p = Problem([rows, rows, rows], [500, 320, 128], 2, 2, 64, mode, g, "bf16", 64, seed=40, garbage=False)
    v = (qm.dequantize(p.cache.value, torch.float32) * size).bfloat16()
    for b, i in ((0, 2), (0, 3), (1, 0), (1, 4), (2, 0), (2, 1)):
        v[p.table_host[b, i]] = 0
    p.cache = qm.KVCache(p.cache.key, qm.quantize(v.contiguous(), g, 4, mode))
    p.table_host[0, 5], p.table_host[1, 2] = -1, p.cache.pages
    p.table = torch.from_numpy(p.table_host).to(DEV)
    got = p.call()
    assert qm.last_path() == ("kv_attention_prompt" if rows == 300 else "kv_attention_rows")
    p.check(got)
    assert (got[2 * rows :] == 0).all()
