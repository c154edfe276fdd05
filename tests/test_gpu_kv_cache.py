"""Rows into a 4-bit cache and back on the GPU, against the CPU oracle of quantization: bytes equal, numbers equal."""
import numpy as np
import pytest
import torch

import kv_reference as ref
import oracle
from helpers import ORACLE_DT, to_oracle

pytestmark = pytest.mark.gpu

qm = pytest.importorskip("quantized_matmul_amd")

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def rand(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + 0.1).to(DTYPES[dtype]).to(DEV)


def parts(cache):
    return [t for w in (cache.key, cache.value) for t in (w.value, w.scales, w.biases)]


def at(t, slots, page):
    """Rows [T, heads, ...] of a pool."""
    s = slots.long().cpu()
    return t[s // page, :, s % page] if t is not None else None


CASES = [
    # T, H, D, mode, g, dtype, page
    (1, 8, 128, "affine", 64, "bf16", 16),
    (8, 1, 32, "affine", 32, "f32", 16),
    (37, 3, 64, "affine", 64, "f16", 48),
    (100, 2, 256, "affine", 128, "bf16", 16),
    (51, 5, 96, "mxfp4", 32, "bf16", 32),
    (7, 3, 160, "mxfp4", 32, "f32", 16),
    (129, 6, 192, "nvfp4", 16, "f16", 64),
    (65, 1, 96, "nvfp4", 16, "bf16", 16),
    (2100, 8, 128, "affine", 64, "bf16", 64),      # runs of words in a thread
    (2100, 8, 128, "nvfp4", 16, "f32", 112),
    (5003, 3, 224, "mxfp4", 32, "f16", 64),
    (2500, 4, 128, "affine", 32, "f32", 16),
]


@pytest.mark.parametrize("T,H,D,mode,g,dtype,page", CASES)
def test_write_and_read(T, H, D, mode, g, dtype, page):
    print(f"cache T{T} H{H} D{D} {mode} g{g} {dtype} page {page}", flush=True)
    pages = -(-T // page) + 2
    cache = qm.kv_cache(pages, H, page, D, g, mode, DTYPES[dtype], DEV)
    for t in parts(cache):
        if t is not None:
            t.copy_((torch.arange(t.numel(), device=DEV) * 7919 % 120).view(t.shape).to(t.dtype))   # marks
    before = [None if t is None else t.clone() for t in parts(cache)]
    order = torch.randperm(pages * page, generator=torch.Generator().manual_seed(T))[:T].to(torch.int32)
    left_out = torch.arange(T) % 7 == 3
    slots = torch.where(left_out, torch.tensor([-1, pages * page, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32)[torch.arange(T) % 4], order)
    row = rand((T, 2 * H + 1, D), dtype, D + T)
    k, v = row[:, :H], row[:, H + 1 :]                 # 16-byte aligned rows that lie apart
    qm.kv_cache_write(cache, k, v, slots.to(DEV))
    kept = slots[~left_out]
    for side, x in ((0, k), (3, v)):
        words, scales, biases = oracle.quantize(to_oracle(x[(~left_out).to(DEV)]).reshape(-1, D), ORACLE_DT[DTYPES[dtype]], g, 4, mode)
        for t, want in zip(parts(cache)[side : side + 3], (words, scales, biases)):
            if t is not None:
                np.testing.assert_array_equal(to_oracle(at(t.cpu(), kept, page)).reshape(want.shape), want)
    # everything else is as it was
    hit = torch.zeros(pages * page, dtype=torch.bool)
    hit[kept.long()] = True
    hit = hit.view(pages, page)[:, None, :, None].to(DEV)
    for t, b in zip(parts(cache), before):
        if t is not None:
            assert torch.equal(torch.where(hit, b, t), b)
    # back as numbers: dequantize's, in every type; twice the same slot, none, zeros
    for out in DTYPES.values():
        ask = torch.cat([slots, kept.flip(0), kept[:1]])
        got = qm.kv_cache_read(cache, ask.to(DEV), dtype=out)
        for side, w, y in ((0, cache.key, got[0]), (3, cache.value, got[1])):
            dense = qm.dequantize(w, out)
            inside = (ask >= 0) & (ask < pages * page)
            want = at(dense.cpu(), torch.where(inside, ask, 0), page)
            want[~inside] = 0
            assert torch.equal(y.cpu(), want)
    # and those are the numbers that the codes stand for
    w = cache.key
    scales = w.scales.cpu().double().numpy() if mode == "affine" else w.scales.cpu().numpy()
    num = ref.values(w.value.cpu().numpy(), scales, None if w.biases is None else w.biases.cpu().double().numpy(), mode, g)
    got = qm.kv_cache_read(cache, kept.to(DEV), dtype=torch.float32)[0].cpu().double().numpy()
    want = at(torch.from_numpy(num), kept, page).numpy()
    assert (np.abs(got - want) <= 2.0 ** -24 * np.abs(want)).all()


@pytest.mark.parametrize("mode,g", [("affine", 32), ("nvfp4", 16), ("mxfp4", 32)])
def test_rows_at_odd_addresses(mode, g):
    """Rows whose address or stride is no multiple of 16 bytes give the bytes that aligned ones give."""
    T, H, D = 33, 3, 64
    flat = rand((T * (2 * H * D + 5) + 3,), "bf16", 4)
    k = flat.as_strided((T, H, D), (2 * H * D + 5, D, 1), 3)
    v = flat.as_strided((T, H, D), (2 * H * D + 5, D, 1), 3 + H * D)
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    a, b = (qm.kv_cache(3, H, 16, D, g, mode, torch.bfloat16, DEV) for _ in range(2))
    qm.kv_cache_write(a, k, v, slots)
    qm.kv_cache_write(b, k.contiguous(), v.contiguous(), slots)
    for x, y in zip(parts(a), parts(b)):
        assert x is None or torch.equal(x, y)
    qm.kv_cache_write(a, k[:1].expand(T, H, D), v[:1].expand(T, H, D), slots)          # one row for all
    qm.kv_cache_write(b, k[:1].expand(T, H, D).contiguous(), v[:1].expand(T, H, D).contiguous(), slots)
    for x, y in zip(parts(a), parts(b)):
        assert x is None or torch.equal(x, y)


def test_constant_and_zero_rows():
    cache = qm.kv_cache(1, 1, 16, 64, 32, "affine", torch.bfloat16, DEV)
    k = torch.tensor([0.0, 1.5, -2.0], device=DEV, dtype=torch.bfloat16)[:, None, None].expand(3, 1, 64).contiguous()
    qm.kv_cache_write(cache, k, -k, torch.tensor([2, 0, 9], dtype=torch.int32, device=DEV))
    a, b = qm.kv_cache_read(cache, torch.tensor([2, 0, 9, 3], dtype=torch.int32, device=DEV))
    assert torch.equal(a[:3], k) and torch.equal(b[:3], -k) and (a[3] == 0).all()
    for mode in ("mxfp4", "nvfp4"):
        cache = qm.kv_cache(1, 1, 16, 64, mode=mode, device=DEV)
        qm.kv_cache_write(cache, k, -k, torch.tensor([2, 0, 9], dtype=torch.int32, device=DEV))
        a, b = qm.kv_cache_read(cache, torch.tensor([2, 0, 9], dtype=torch.int32, device=DEV))
        # nvfp4: 2 / 6 is held as the nearest e4m3, 11/32, and six of those are 2.0625; 1.5 / 6 is one itself
        want = k * torch.tensor([1, 1, 2.0625 / 2 if mode == "nvfp4" else 1], device=DEV, dtype=k.dtype)[:, None, None]
        assert torch.equal(a.bfloat16(), want) and torch.equal(b.bfloat16(), -want)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("mode,g", [("affine", 32), ("affine", 64), ("affine", 128), ("mxfp4", 32), ("nvfp4", 16)])
def test_ties_zeros_and_small_rows(mode, g, dtype):
    """Quotients half way between codes, signed zeros in either order, the smallest and the largest groups: the oracle's bytes."""
    D, rows = 128, []
    step = torch.arange(D).float()
    for size in (1.0, 0.25, 2.0 ** -12, 3.0):
        rows += [step % 31 / 2 * size, (step % 31 / 2 - 7.5) * size, (step % 13 / 4 - 1.5) * size, (step * 7 % 25 / 8 - 1.5) * size]
    zeros = torch.zeros(D)
    rows += [zeros, -zeros, torch.where(step % 3 == 0, -zeros, zeros), torch.where(step % 5 == 1, -zeros, zeros),
             torch.where(step % 4 == 0, -zeros, step % 4), torch.where(step % 4 == 0, zeros, -(step % 4)),
             torch.where(step % 32 < 16, zeros, -zeros), torch.where(step % 32 < 16, -zeros, zeros)]
    tiny, most = torch.finfo(DTYPES[dtype]).smallest_normal, torch.finfo(DTYPES[dtype]).max
    rows += [(step % 9 - 4) * tiny, (step % 9 - 4) * tiny / 8, step * tiny, (step % 17 - 8) / 8 * most / 8, torch.full((D,), -tiny)]
    x = torch.stack(rows).to(DTYPES[dtype])[:, None].to(DEV)
    cache = qm.kv_cache(2, 1, 32, D, g, mode, DTYPES[dtype], DEV)
    slots = torch.arange(len(rows), dtype=torch.int32, device=DEV)
    qm.kv_cache_write(cache, x, x.flip(0), slots)
    for w, y in ((cache.key, x), (cache.value, x.flip(0))):
        want = oracle.quantize(to_oracle(y).reshape(-1, D), ORACLE_DT[DTYPES[dtype]], g, 4, mode)
        for t, ref_t in zip((w.value, w.scales, w.biases), want):
            if t is not None:
                np.testing.assert_array_equal(to_oracle(at(t.cpu(), slots.cpu(), 32)).reshape(ref_t.shape), ref_t)


def test_a_pool_past_32_bits():
    """A pool of more than 2^32 bytes of codes: its last rows are written and read where they lie."""
    H, D, page = 8, 256, 4096
    pages = (1 << 32) // (H * page * D // 2) + 2
    cache = qm.kv_cache(pages, H, page, D, 128, "affine", torch.bfloat16, DEV)
    slots = torch.tensor([pages * page - 1, 0, (pages - 1) * page, pages * page // 2], dtype=torch.int32, device=DEV)
    k, v = rand((4, H, D), "bf16", 5), rand((4, H, D), "bf16", 6)
    qm.kv_cache_write(cache, k, v, slots)
    small = qm.kv_cache(1, H, 16, D, 128, "affine", torch.bfloat16, DEV)
    near = torch.arange(4, dtype=torch.int32, device=DEV)
    qm.kv_cache_write(small, k, v, near)
    for a, b in zip(qm.kv_cache_read(cache, slots), qm.kv_cache_read(small, near)):
        assert torch.equal(a, b)
    assert int((cache.key.value != 0).any(-1).sum()) <= 4 * H


@pytest.mark.parametrize("mode", ["affine", "mxfp4"])
def test_captured_on_another_stream_and_replayed(mode):
    """Rows turned, written and read back, and a gradient turned back, in one graph: every replay gives the eager bits
    for what its buffers hold then."""
    D, T = 64, 300
    freqs = qm.rotary_frequencies(D, device=DEV)
    x, v = [rand((T, 2, D), "bf16", i) for i in range(2)]
    positions = torch.arange(T, dtype=torch.int32, device=DEV)
    slots = torch.randperm(20 * 16, generator=torch.Generator().manual_seed(5))[:T].to(torch.int32).to(DEV)

    def run(cache, turned):
        qm.rotary(x, positions, freqs, out=turned)
        qm.kv_cache_write(cache, turned, v, slots)
        return (*qm.kv_cache_read(cache, slots), qm.rotary_grad(v, positions, freqs))

    cache, turned, stream = qm.kv_cache(20, 2, 16, D, mode=mode, device=DEV), torch.empty_like(x), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run(cache, turned)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs = run(cache, turned)
    torch.cuda.current_stream().wait_stream(stream)
    for i in range(4):
        x.copy_(rand((T, 2, D), "bf16", 10 + i))
        positions.add_(i)
        slots.copy_(slots.roll(1))
        other = qm.kv_cache(20, 2, 16, D, mode=mode, device=DEV)
        want = run(other, torch.empty_like(x))
        (torch.randn(1 << 16, device=DEV) * 2.0).sum()      # unrelated work
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), i


def test_refusals():
    cache = qm.kv_cache(2, 2, 16, 64, 64, "affine", torch.bfloat16, DEV)
    k, slots = rand((3, 2, 64), "bf16", 1), torch.zeros(3, dtype=torch.int32, device=DEV)
    for bad in (lambda: qm.kv_cache_write(cache, k, k[:2], slots), lambda: qm.kv_cache_write(cache, k, k, slots[:2]),
                lambda: qm.kv_cache_write(cache, k.half(), k.half(), slots), lambda: qm.kv_cache_write(cache, k, k, slots.long()),
                lambda: qm.kv_cache_write(cache, k.transpose(0, 1), k.transpose(0, 1), slots),
                lambda: qm.kv_cache_write(cache, k[..., ::2], k, slots), lambda: qm.kv_cache_write(cache, k.cpu(), k, slots),
                lambda: qm.kv_cache_read(cache, slots.cpu()), lambda: qm.kv_cache_read(cache, slots, dtype=torch.int32),
                lambda: qm.kv_cache(2, 2, 16, 100, 64), lambda: qm.KVCache(cache.key, qm.kv_cache(2, 2, 16, 64, mode="nvfp4", device=DEV).value),
                lambda: qm.KVCache(cache.key, qm.kv_cache(3, 2, 16, 64, 64, device=DEV).value),
                lambda: qm.KVCache(qm.quantize(k, 64, 4), qm.quantize(k, 64, 4))):
        with pytest.raises(ValueError):
            bad()
    for make in (lambda: qm.kv_cache(2, 2, 24, 64, 64), lambda: qm.kv_cache(2, 2, 16, 64, 16),
                 lambda: qm.kv_cache(2, 2, 16, 48, 16, "nvfp4"), lambda: qm.kv_cache(1, 1, 16, 288, 32)):
        with pytest.raises(qm.QlinError):
            c = make()
            qm.kv_cache_read(c, slots, dtype=torch.float32)
    w = qm.quantize(rand((2, 2, 16, 64), "bf16", 3), 64, 8)
    with pytest.raises((qm.QlinError, ValueError)):
        qm.kv_cache_read(qm.KVCache(w, w), slots)
