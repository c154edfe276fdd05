"""Attention over a 4-bit cache on the GPU: what the matrix cores' 16-bit operands may cost. Problems and formulas are those
of test_gpu_kv_attention, tolerances narrower where a rounding is left out."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from test_gpu_kv_attention import DEV, DTYPES, UNIT, Problem, f64, rand

pytestmark = pytest.mark.gpu

qm = pytest.importorskip("quantized_matmul_amd")


def bound(p, window, pv, codes, causal=True):
    """What attention has to give, and how far off it may be: test_gpu_kv_attention's terms, with p and values rounded to pv
    each (codes: p times the scale, which multiplies c - 8) and keys that are exact."""
    pools, q, first = p.dense(), f64(p.q), 0
    out, tol, u = np.zeros(q.shape), np.zeros(q.shape), UNIT[p.dtype]
    for b, (n, L) in enumerate(zip(p.rows, p.lengths_host)):
        i = np.arange(L)
        k, v = [x[p.table_host[b, i // p.page], :, i % p.page] for x in pools]
        rows = slice(first, first + n)
        o, size, _ = ref.attention(q[rows], k, v, n, p.D ** -0.5, causal, window)
        if codes:
            s = np.repeat(f64(p.cache.value.scales), p.g, -1)[p.table_host[b, i // p.page], :, i % p.page]
            rounded = ref.attention(q[rows], k, v, n, p.D ** -0.5, causal, window, None, 8 * s)[1] * pv
        else:
            rounded = 2 * size * pv
        d = 4 * np.sqrt(p.D) * 2.0 ** -24 * p.D ** -0.5 * np.abs(q[rows]).sum(-1, keepdims=True) * 6 * np.abs(k).max()
        out[rows] = o
        tol[rows] = rounded + size * (2 * d + 2.0 ** -22 + (np.sqrt(L) + 8) * 2.0 ** -24) + u * np.abs(o) \
            + 2.0 ** -24 * np.abs(v).max() + (2.0 ** -24 if p.dtype == "f16" else 0)
        first += n
    return out, tol


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


@pytest.mark.parametrize("power", [10, 20, 40, 60])
@pytest.mark.parametrize("order", ["down", "up"])
@pytest.mark.parametrize("D,g,G", [(128, 32, 1), (128, 64, 1), (64, 32, 20), (256, 64, 3), (128, 128, 2)])
def test_small_values_that_take_all_the_weight_beside_large_ones(D, g, G, order, power):
    """Tokens whose weight lies on values that are 2^-power of others, whose keys they turn away from."""
    print(f"weights {order} 2^{power} D{D} g{g} G{G}", flush=True)
    p = Problem([1, 1], [630, 400], 1, G, D, "affine", g, "bf16", 64, seed=48, garbage=False)    # one workgroup each
    p.q = (p.q[:, :1] + 0.1 * p.q).bfloat16()                # the heads of a token look the same way
    k, v = [qm.dequantize(w, torch.float32) for w in (p.cache.key, p.cache.value)]
    for b in range(2):
        n = -(-p.lengths_host[b] // 64)
        large = [i for i in range(n) if ((i * 5 // n) % 2 == 0) == (order == "down")]
        at = torch.from_numpy(p.table_host[b, large].astype(np.int64)).to(DEV)
        away = p.q[b].float().mean(0)
        k[at] = -away * (150 * D ** 0.5 / (away * away).sum()) + 0.02 * k[at]
        small = torch.ones(v.shape[0], dtype=torch.bool, device=DEV)
        small[at] = False
        mine = torch.zeros_like(small)
        mine[torch.from_numpy(p.table_host[b, :n].astype(np.int64)).to(DEV)] = True
        v[small & mine] *= 2.0 ** -power
    p.cache = qm.KVCache(*[qm.quantize(x.bfloat16().contiguous(), g, 4) for x in (k, v)])
    got = p.call()
    assert qm.last_path() == "kv_attention_rows"
    want, tol = bound(p, 0, 2.0 ** -11, False)
    values = np.abs(p.dense()[1])
    for b in range(2):
        mine = p.table_host[b, : -(-p.lengths_host[b] // 64)]
        largest = values[mine].max()
        low = np.min([values[i].max() for i in mine])        # the small pages' largest
        # of the large keys e^-120 is left; what is small in a page keeps 2^-19 of its largest, |z| + 15 s up to 3 of those
        tol[b] += -2.0 ** -24 * largest + 3 * 2.0 ** -18 * low + 2.0 ** -160 * largest
    err = np.abs(f64(got) - want)
    assert np.isfinite(f64(got)).all() and (np.abs(want).max() < 100 * low)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("D,g,G", [(64, 32, 2), (64, 64, 4), (96, 32, 1), (128, 64, 2), (128, 128, 4), (192, 64, 1), (256, 64, 1)])
def test_weights_of_values_as_codes(D, g, G, rows):
    """bf16 tokens: what p times a group's scale, which multiplies its codes, loses does not show beside the output's rounding.

    Rounded to f16 it is off by 2^-11 / sqrt(3) of p s |c - 8| in the mean square, independent for each key; p s |c - 8| is
    about p |v| here (values around zero), whose squares' sum is at most max |v| |o| where few keys hold the weight. The
    output's rounding to bf16 is off by 2^-9 / sqrt(3) of it and more: a quarter at most, and sqrt(1 + 1 / 16) = 1.03 of
    it in all; 1.1 leaves room for |v| above |o|."""
    print(f"codes D{D} g{g} G{G} rows {rows}", flush=True)
    p = Problem([rows] * 12, [40 + 37 * i for i in range(12)], 4, G, D, "affine", g, "bf16", 16, seed=49, std=2.5, garbage=False)
    got = p.call()
    assert qm.last_path() == "kv_attention_rows"
    want, _ = bound(p, 0, 0.0, False)
    rounding = f64(torch.from_numpy(want).bfloat16()) - want
    off = np.sqrt(((f64(got) - want) ** 2).mean() / (rounding ** 2).mean())
    print(f"error over that of rounding: {off:.3f}")
    assert off <= 1.1


@pytest.mark.parametrize("D,g", [(64, 32), (96, 32), (128, 64), (128, 128), (192, 64), (256, 32)])
def test_prompts_of_f16_keep_their_keys(D, g):
    """f16 prompts over affine keys: scores as exact as fp32 sums, though a key has more bits than f16.

    What is rounded to f16 then is p, a value and the output, each as much as the other: sqrt(3) of the output's rounding in
    the mean square, where one key holds the weight, and less elsewhere."""
    print(f"f16 prompt D{D} g{g}", flush=True)
    p = Problem([290, 600], [700, 600], 1, 2, D, "affine", g, "f16", 64, seed=50, std=2.0, garbage=False)
    got = p.call()
    assert qm.last_path() == "kv_attention_prompt"
    want, tol = bound(p, 0, 2.0 ** -11, False)
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), (err / tol).max()
    rounding = f64(torch.from_numpy(want).half()) - want
    off = np.sqrt((err ** 2).mean() / (rounding ** 2).mean())
    print(f"error over that of rounding: {off:.3f}")
    assert off <= 3 ** 0.5
