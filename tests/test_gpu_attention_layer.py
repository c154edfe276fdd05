"""The example attention layer: the operators around a 4-bit cache run together, prompts and tokens, eagerly and as a
captured step.

Each operator is compared with its 64-bit statement fed the kernels' own intermediate values: rotated rows of the bf16
projection round once (2^-8 of the value; angles of positions below 2^10 are off by 2^-24 of themselves in fp32
frequencies, which both sides take, and sin and cos by less than 2^-20), the cache holds what `quantize` makes of those
rows, and attention keeps test_gpu_kv_attention's bounds over what the cache holds."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import kv_reference as ref
from test_gpu_kv_attention import Problem

pytestmark = pytest.mark.gpu

qm = pytest.importorskip("quantized_matmul_amd")

DEV = "cuda:0"


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer_example", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def f64(t):
    return t.detach().cpu().double().numpy()


def rows(n, D, seed):
    return torch.randn(n, D, generator=torch.Generator().manual_seed(seed)).bfloat16().to(DEV)


def bounds(cache, mode, g, requests, counts, q, heads):
    """A problem of test_gpu_kv_attention over what this cache holds."""
    p = Problem.__new__(Problem)
    p.rows, p.lengths_host, p.H, p.D, p.dtype = counts, requests.lengths_host, cache.heads, cache.head_dim, "bf16"
    p.page, p.mode, p.g, p.cache, p.q = cache.page_size, mode, g, cache, q
    p.table_host = requests.table_host.numpy()
    return p


@pytest.mark.parametrize("mode,g", [("affine", 64), ("mxfp4", 32), ("nvfp4", 16)])
def test_prompts_then_tokens(example, mode, g):
    """Two steps of ragged prompts, one of them for some of the requests only, then tokens."""
    layer = example.random_layer(256, 8, 2, 64)
    requests = example.Requests(3, 700, 16, DEV)
    cache = qm.kv_cache(requests.pages, 2, 16, 64, g, mode, device=DEV)
    for step, counts in enumerate(([150, 7, 400], [33, 0, 1], [1, 1, 1], [1, 1, 1])):
        print(f"layer {mode} step {counts}", flush=True)
        T = sum(counts)
        positions, slots, lengths, offsets = [t.to(DEV) for t in requests.add(counts)]
        x = rows(T, 256, step)
        plain = f64(qm.quantized_matmul(x, layer.w_in)).reshape(T, 12, 64)
        q, k, v = layer.project(x, positions)
        want = ref.rotary(plain[:, :10], f64(positions).astype(np.int64), f64(layer.freqs))
        size = np.abs(plain[:, :10])
        size = size + np.roll(size, 32, -1)
        for got, want in ((q, want[:, :8]), (k, want[:, 8:])):
            assert (np.abs(f64(got) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size[:, :8].max()).all()
        assert (f64(v) == plain[:, 10:]).all()
        y = layer.forward(x, cache, positions, slots, requests.table, lengths, offsets)
        for got, row in zip(qm.kv_cache_read(cache, slots, torch.bfloat16), (k, v)):
            made = qm.quantize(row.contiguous(), g, 4, mode)
            assert torch.equal(got, qm.dequantize(made, torch.bfloat16))
        o = qm.kv_cache_attention(q, cache, requests.table, lengths, offsets)
        bounds(cache, mode, g, requests, counts, q, 8).check(o)
        assert torch.equal(y, qm.quantized_matmul(o.view(T, -1), layer.w_out))


@pytest.mark.parametrize("mode", ["affine", "nvfp4"])
def test_captured_token_steps(example, mode):
    """A replayed step gives the bits of the eager one, the cache's among them, with other work between the replays."""
    layer = example.random_layer(256, 8, 2, 64)
    made = []
    for captured in (False, True):
        requests = example.Requests(4, 500, 16, DEV)
        cache = qm.kv_cache(requests.pages, 2, 16, 64, mode=mode, device=DEV)
        positions, slots, lengths, offsets = [t.to(DEV) for t in requests.add([200, 1, 60, 3])]
        layer.forward(rows(264, 256, 1), cache, positions, slots, requests.table, lengths, offsets)
        step = example.TokenStep(layer, cache, requests) if captured else None
        outs = []
        for i in range(5):
            positions, slots, lengths, _ = requests.add([1] * 4)
            x = rows(4, 256, 10 + i)
            if captured:
                outs.append(step(x, positions, slots, lengths).clone())
            else:
                outs.append(layer.forward(x, cache, positions.to(DEV), slots.to(DEV), requests.table, lengths.to(DEV)))
            (torch.randn(1 << 16, device=DEV) * 2.0).sum()      # unrelated work
            torch.cuda.synchronize()
        made.append(outs + [t for w in (cache.key, cache.value) for t in (w.value, w.scales)])
    for eager, replayed in zip(*made):
        assert torch.equal(eager, replayed)


def test_the_example_runs(example):
    y = example.main(["--requests", "3", "--prompt", "100", "--tokens", "4", "--dim", "256", "--heads", "4",
                      "--key-heads", "2", "--mode", "mxfp4"])
    assert y.shape == (3, 256) and torch.isfinite(y).all()
