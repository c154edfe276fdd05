"""Attention over a 4-bit cache on the GPU against kv_reference in 64 bits.

Tolerance, for each output o = sum p v with size = sum p |v|:
  scores    the products of codes and q are exact; sums of D of them, offset by 16, and of the groups round in fp32: 4
            sqrt(D) roundings of 2^-24 (their signs are random, 4 standard deviations) of scale * sum |q| (31 s + |z|),
            which is below 40 * scale * sum |q| * max |k| for affine codes (s is 1/15 of a group's range, at most 2/15 of
            max |k|: 31 s <= 4.2 max |k|; taken as 6); p then is off by e^d, output and sum alike: 2 d of the size.
            In prompts u is f16's for either type, and what is small beside the largest value is held to 2^-24 of that.
  keys      in prompts rounded to f16 for either type: independent errors of at most 2^-11 |k|, 2^-11 / sqrt(3) |k| in
            their standard deviation (2^-25 of the largest where f16 has no more bits, inside the scores' bound); through scores and softmax they reach o as `spread` of kv_reference, times 6 for the many outputs
            (and twice that, as p and the sum of p move together).
  exp2      1 ulp each: 2 * 2^-23.
  p, v      on the matrix cores each rounded to the type once: 2 u of the size, u = eps / 2 of the type. Where the values
            stay codes (bf16, affine) p times the group's scale is rounded instead, and multiplies c - 8, the rest being
            fp32: u p s |c - 8|, which is at most 8 s u p for each key. (Other bf16 affine values and their p are
            rounded to f16, inside this.)
  sums      fp32 over L keys: sqrt(L) + 8 roundings of 2^-24.
  output    one rounding: u of itself; and f16's smallest step.
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


def f64(t):
    return t.detach().cpu().double().numpy()


def rand(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(DTYPES[dtype]).to(DEV)


class Problem:
    """Sequences of given rows and lengths in a pool of shuffled pages, and what attention has to give."""

    def __init__(self, rows, lengths, H, G, D, mode, g, dtype, page, seed=0, std=1.5, spare=2, garbage=True):
        self.rows, self.lengths_host, self.H, self.G, self.D, self.dtype = rows, lengths, H, G, D, dtype
        self.page, self.mode, self.g = page, mode, g
        need = [-(-n // page) for n in lengths]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
        kv = [rand((pages, H, page, D), dtype, seed + 1 + i) + 0.1 for i in range(2)]
        self.cache = qm.KVCache(*[qm.quantize(x, g, 4, mode) for x in kv])
        self.table_host = np.full((len(lengths), max(max(need, default=0), 1)), -1, dtype=np.int32)
        used = np.zeros((pages, page), dtype=bool)
        for b, n in enumerate(need):
            mine, order = order[:n], order[n:]
            self.table_host[b, :n] = mine
            for i in range(lengths[b]):
                used[mine[i // page], i % page] = True
        if garbage and mode == "affine":      # what lies behind a sequence's end is no number at all
            hole = torch.from_numpy(~used).to(DEV)[:, None, :, None]
            for w in (self.cache.key, self.cache.value):
                w.scales.masked_fill_(hole, float("nan"))
                w.biases.masked_fill_(hole, float("inf"))
        elif garbage:
            hole = torch.from_numpy(~used).to(DEV)[:, None, :, None]
            for w in (self.cache.key, self.cache.value):
                w.scales.masked_fill_(hole, 255)          # NaN in both
        self.q = rand((sum(rows), H * G, D), dtype, seed + 7, std)
        self.table = torch.from_numpy(self.table_host).to(DEV)
        self.lengths = torch.tensor(lengths, dtype=torch.int32, device=DEV)
        starts = np.concatenate([[0], np.cumsum(rows)])
        self.offsets = torch.tensor(starts, dtype=torch.int32, device=DEV)

    def dense(self):
        out = []
        for w in (self.cache.key, self.cache.value):
            scales = f64(w.scales) if self.mode == "affine" else w.scales.cpu().numpy()
            out.append(ref.values(w.value.cpu().numpy(), scales, None if w.biases is None else f64(w.biases), self.mode, self.g))
        return out

    def want(self, scale=None, causal=True, window=0, rows=None):
        scale = self.D ** -0.5 if scale is None else scale
        pools, q, first = self.dense(), f64(self.q), 0
        out, tol = np.zeros(q.shape), np.zeros(q.shape)
        u = UNIT[self.dtype]
        for b, (n, L) in enumerate(zip(self.rows, self.lengths_host)):
            i = np.arange(L)
            p = self.table_host[b, i // self.page] if L else i
            dead = (p < 0) | (p >= pools[0].shape[0])
            k, v = [np.where(dead[:, None, None], 0.0, x[np.where(dead, 0, p), :, i % self.page]) for x in pools] if L else \
                (np.zeros((0, self.H, self.D)),) * 2
            o, size, spread = ref.attention(q[first : first + n], k, v, n, scale, causal, window, dead)
            if self.mode == "affine" and self.dtype == "bf16" and not self.prompt and L:
                s = np.repeat(np.nan_to_num(f64(self.cache.value.scales)), self.g, -1)
                steps = 8 * np.where(dead[:, None, None], 0.0, s[np.where(dead, 0, p), :, i % self.page])
                size = size + ref.attention(q[first : first + n], k, v, n, scale, causal, window, dead, steps)[1]
            kmax = np.abs(k).max() if L else 0.0
            d = 4 * np.sqrt(self.D) * 2.0 ** -24 * abs(scale) * np.abs(q[first : first + n]).sum(-1, keepdims=True) * 6 * kmax
            out[first : first + n] = o
            pv = 2.0 ** -11 if self.prompt else u
            tol[first : first + n] = size * (2 * pv + 2 * d + 2.0 ** -22 + (np.sqrt(L) + 8) * 2.0 ** -24) + u * np.abs(o) \
                + (2.0 ** -24 if self.dtype == "f16" else 0)
            if self.prompt and self.mode == "affine":
                tol[first : first + n] += 12 * 2.0 ** -11 / np.sqrt(3) * spread
            if self.prompt and L:
                tol[first : first + n] += 2.0 ** -24 * np.abs(v).max()
            first += n
        return out, tol

    def call(self, **how):
        return qm.kv_cache_attention(self.q, self.cache, self.table, self.lengths, offsets=self.offsets, **how)

    def check(self, got, **how):
        self.prompt = qm.last_path() == "kv_attention_prompt"
        want, tol = self.want(**how)
        err = np.abs(f64(got) - want)
        assert np.isfinite(f64(got)).all()
        assert (err <= tol).all(), (err.max(), (err / np.maximum(tol, 1e-30)).max(), np.unravel_index((err - tol).argmax(), err.shape))


FORMATS = [("affine", 32), ("affine", 64), ("affine", 128), ("mxfp4", 32), ("nvfp4", 16)]
SIZES = [64, 96, 128, 192, 256]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("mode,g", FORMATS)
@pytest.mark.parametrize("D", SIZES + [32, 160])
def test_one_row_each(D, mode, g, dtype):
    """Decode: a row a sequence; lengths of none, one, around a run, a step, a workgroup's step and chunks."""
    if D % g:
        pytest.skip("head_dim is no multiple of the group")
    print(f"decode D{D} {mode} g{g} {dtype}", flush=True)
    lengths = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 100, 127, 128, 129, 300, 513]
    p = Problem([1] * len(lengths), lengths, 2, 3, D, mode, g, dtype, 16, seed=D + g)
    got = p.call()
    p.check(got)
    assert torch.equal(got, qm.kv_cache_attention(p.q, p.cache, p.table, p.lengths))      # offsets say nothing new
    assert qm.last_path() == ("kv_attention_simple" if dtype == "f32" or D not in SIZES else "kv_attention_rows")
    assert (got[0] == 0).all()


@pytest.mark.parametrize("H,G", [(1, 1), (8, 4), (1, 16), (2, 17), (1, 33), (3, 8), (5, 5)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_head_layouts(H, G, dtype):
    p = Problem([1, 1, 1], [70, 257, 1], H, G, 128, "affine", 64, dtype, 32, seed=H * 100 + G)
    p.check(p.call())
    p = Problem([3, 1, 6], [70, 257, 9], H, G, 64, "mxfp4", 32, dtype, 32, seed=H * 100 + G)
    p.check(p.call())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("mode,g", FORMATS)
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 40), (False, 0), (False, 33)])
def test_rows_of_several_tokens(mode, g, dtype, causal, window):
    """Drafted tokens and short prompts: rows that see few keys or none (more rows than keys), empty sequences."""
    print(f"rows {mode} g{g} {dtype} causal {causal} window {window}", flush=True)
    rows, lengths = [1, 5, 0, 7, 3, 40, 2, 0, 4], [90, 200, 60, 3, 0, 40, 129, 0, 161]
    p = Problem(rows, lengths, 2, 2, 128, mode, g, dtype, 48, seed=g)
    p.check(p.call(causal=causal, window=window), causal=causal, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("mode,g", FORMATS)
@pytest.mark.parametrize("D", SIZES)
def test_prompts(D, mode, g, dtype):
    """Many rows of a sequence, with keys before them and without, of odd numbers."""
    if D % g:
        pytest.skip("head_dim is no multiple of the group")
    print(f"prompt D{D} {mode} g{g} {dtype}", flush=True)
    p = Problem([150, 331, 77], [400, 331, 1000], 1, 3, D, mode, g, dtype, 64, seed=D + g)
    p.check(p.call())
    assert qm.last_path() == "kv_attention_prompt"


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 100), (False, 0), (False, 70)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_prompt_masks(dtype, causal, window):
    for rows, lengths, page in (([200, 1, 300], [260, 500, 120], 16), ([513], [513], 80), ([260, 0, 270], [0, 10, 100], 16),
                                ([600, 1, 700], [660, 500, 720], 16), ([760, 0, 870], [0, 10, 300], 32)):
        p = Problem(rows, lengths, 2, 2, 128, "affine", 64, dtype, page, seed=len(rows))
        p.check(p.call(causal=causal, window=window), causal=causal, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 3, 90, 300])
def test_bad_pages_take_their_keys_out(dtype, rows):
    p = Problem([rows, rows], [400, 170], 2, 2, 64, "affine", 64, dtype, 16, seed=5)
    for b, i, v in ((0, 0, -1), (0, 3, 1 << 30), (0, 9, -(1 << 31)), (1, 2, p.cache.pages), (1, 10, -5)):
        p.table_host[b, i] = v
    p.table = torch.from_numpy(p.table_host).to(DEV)
    p.check(p.call())
    p.table_host[1, :] = -1                     # nothing is there at all
    p.table = torch.from_numpy(p.table_host).to(DEV)
    got = p.call()
    p.check(got)
    assert (got[rows:] == 0).all()


def test_pages_may_be_shared_and_long_tables_end_early():
    p = Problem([1, 1], [200, 200], 2, 2, 128, "affine", 64, "bf16", 16, seed=6)
    p.table_host[1, :6] = p.table_host[0, :6]   # a common prefix
    wide = np.full((2, 100), 1 << 20, dtype=np.int32)
    wide[:, :13] = p.table_host
    p.table_host, p.table = wide, torch.from_numpy(wide).to(DEV)
    p.check(p.call())


@pytest.mark.parametrize("rows", [1, 60, 600])
def test_rows_behind_the_last_sequence_stay(rows):
    """A padded batch: rows before the first sequence and behind the last are left as they are."""
    p = Problem([rows, 2], [100, 50], 2, 2, 128, "mxfp4", 32, "bf16", 16, seed=7)
    T = p.q.shape[0]
    q = torch.cat([rand((3, 4, 128), "bf16", 1), p.q, torch.full((5, 4, 128), float("nan"), device=DEV, dtype=torch.bfloat16)])
    out = torch.full((T + 8, 4, 128), 7.0, device=DEV, dtype=torch.bfloat16)
    got = qm.kv_cache_attention(q, p.cache, p.table, p.lengths, offsets=p.offsets + 3, out=out)
    assert got.data_ptr() == out.data_ptr() and (out[:3] == 7).all() and (out[T + 3 :] == 7).all()
    p.check(out[3 : T + 3])         # not by bits: a call's sizes, the padding's among them, choose its kernel
    fresh = qm.kv_cache_attention(q, p.cache, p.table, p.lengths, offsets=p.offsets + 3)
    assert (fresh[:3] == 0).all() and (fresh[T + 3 :] == 0).all()


@pytest.mark.parametrize("rows", [1, 90, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_queries_scale_and_large_scores(rows, dtype):
    p = Problem([rows, rows], [150, 90], 2, 2, 64, "affine", 32, dtype, 16, seed=8)
    wide = torch.randn((2 * rows, 9, 64), device=DEV).to(p.q.dtype)
    wide[:, 3:7] = p.q
    q = wide[:, 3:7]
    got = qm.kv_cache_attention(q, p.cache, p.table, p.lengths, offsets=p.offsets, scale=0.3)
    p.check(got, scale=0.3)
    flat = torch.zeros(2 * rows * 257 + 1, device=DEV, dtype=p.q.dtype)      # rows at odd addresses
    odd = flat.as_strided((2 * rows, 4, 64), (257, 64, 1), 1)
    odd.copy_(p.q)
    assert torch.equal(qm.kv_cache_attention(odd, p.cache, p.table, p.lengths, offsets=p.offsets, scale=0.3), got)
    for scale in (-0.2, 0.0):
        p.check(p.call(scale=scale), scale=scale)
    p.q = (p.q.float() * 40).to(p.q.dtype)      # one key takes all the weight
    got = p.call()
    assert torch.isfinite(got).all()
    p.prompt = qm.last_path() == "kv_attention_prompt"
    want, tol = p.want()
    assert (np.abs(f64(got) - want) <= tol * 4 + 1e-3 * np.abs(want).max()).all()


@pytest.mark.parametrize("rows", [1, 90, 300])
@pytest.mark.parametrize("mode,g", [("affine", 64), ("mxfp4", 32)])
def test_queries_and_keys_of_any_size(rows, mode, g):
    """bf16 reaches far past f16 on both sides: keys of 1e8 under queries of 1e-8, keys of 1e-25, queries of zero."""
    for k_size, q_size in ((1e8, 1e-8), (1e-8, 1e8), (1e-25, 1e-25), (1e-3, 0.0), (1e6, 1e-6)):
        p = Problem([rows, rows], [150, 90], 2, 2, 64, mode, g, "bf16", 16, seed=30)
        live = [qm.dequantize(w, torch.bfloat16) for w in (p.cache.key, p.cache.value)]
        k = torch.nan_to_num(live[0].float(), 0.0, 0.0, 0.0) * k_size
        p.cache = qm.KVCache(qm.quantize(k.bfloat16().contiguous(), g, 4, mode), p.cache.value)
        p.q = (p.q.float() * q_size).bfloat16()
        p.check(p.call())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 90, 300])
def test_values_of_any_size(rows, dtype):
    """Values whose size changes from page to page by powers of two, up and down."""
    p = Problem([rows, rows], [500, 300], 2, 2, 64, "affine", 64, dtype, 64, seed=31, garbage=False)
    v = qm.dequantize(p.cache.value, torch.float32)
    sizes = 2.0 ** torch.tensor([0, 9, -9, 3, -14, 10, -3, 0, 6, -8, 2, -1, 4, 8, -12, 1, 0, 0, 0, 0])[: v.shape[0]]
    p.cache = qm.KVCache(p.cache.key, qm.quantize((v * sizes.to(DEV)[:, None, None, None]).to(DTYPES[dtype]).contiguous(), 64, 4))
    p.check(p.call())
    if dtype == "bf16":
        p.cache = qm.KVCache(p.cache.key, qm.quantize((v * 1e30 * sizes.to(DEV)[:, None, None, None] ** 2).bfloat16().contiguous(), 64, 4))
        p.check(p.call())
        p.cache = qm.KVCache(p.cache.key, qm.quantize((v * 1e-30 * sizes.to(DEV)[:, None, None, None] ** 2).bfloat16().contiguous(), 64, 4))
        p.check(p.call())


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("g", [32, 64])
def test_decoded_values_of_any_size(rows, g):
    """bf16 values that are decoded, of sizes that grow and fall by up to 2^40 from page to page, tiny ones, and zeros.

    They are f16 in units of a power of two of the largest |z| + 15 |s| so far, at most 3 max |v|: what is below 2^-14 of
    it is off by 2^-25 of it, 2^-23 max |v| and less for a weighted mean of values."""
    print(f"decoded sizes rows {rows} g{g}", flush=True)
    p = Problem([rows, rows], [500, 300], 2, 5, 128, "affine", g, "bf16", 64, seed=33, garbage=False)
    v = qm.dequantize(p.cache.value, torch.float32)
    steps = 2.0 ** torch.tensor([0, 18, -20, 3, -14, 20, -3, 0, 16, -8, 2, -1, 4, 8, -12, 1, 0, 0, 0, 0])[: v.shape[0]]
    for size in (1.0, 1e30, 1e-30, 1e-38, 0.0):
        w = (v * size * steps.to(DEV)[:, None, None, None]).bfloat16().contiguous()
        p.cache = qm.KVCache(p.cache.key, qm.quantize(w, g, 4))
        got = p.call()
        assert qm.last_path() == "kv_attention_rows"
        p.prompt = False
        want, tol = p.want()
        tol = tol + 2.0 ** -23 * np.abs(p.dense()[1]).max() + 2.0 ** -126      # (and what bf16 outputs flush or step by)
        assert np.isfinite(f64(got)).all() and (np.abs(f64(got) - want) <= tol).all(), size


def test_long_sequences_in_many_chunks():
    p = Problem([1, 2, 1], [9000, 20000, 4096], 1, 4, 128, "affine", 64, "bf16", 64, seed=9)
    p.check(p.call())
    p.check(p.call(window=5000), window=5000)
    p = Problem([1], [70000], 1, 2, 64, "nvfp4", 16, "f16", 256, seed=10)
    p.check(p.call())
    for rows, lengths, D in (([1, 2], [9000, 20000], 128), ([300, 1], [1500, 1200], 160)):
        p = Problem(rows, lengths, 1, 4, D, "affine", 32, "f32", 64, seed=17)
        p.check(p.call())


def test_a_pool_past_32_bits():
    """Pages that lie past 2^32 bytes of codes."""
    H, D, page = 8, 128, 4096
    pages = (1 << 32) // (H * page * D // 2) + 2
    cache = qm.kv_cache(pages, H, page, D, 64, "affine", torch.bfloat16, DEV)
    L = 5000
    k, v = rand((L, H, D), "bf16", 11), rand((L, H, D), "bf16", 12)
    slots = torch.cat([torch.arange((pages - 1) * page, pages * page), torch.arange((pages - 3) * page, (pages - 3) * page + L - page)])
    qm.kv_cache_write(cache, k, v, slots.to(torch.int32).to(DEV))
    small = qm.kv_cache(2, H, page, D, 64, "affine", torch.bfloat16, DEV)
    qm.kv_cache_write(small, k, v, torch.arange(L, dtype=torch.int32, device=DEV))
    for rows in (1, 70):
        q = rand((rows, 4 * H, D), "bf16", 13)
        lengths = torch.tensor([L], dtype=torch.int32, device=DEV)
        offsets = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
        far = qm.kv_cache_attention(q, cache, torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device=DEV), lengths, offsets)
        near = qm.kv_cache_attention(q, small, torch.tensor([[0, 1]], dtype=torch.int32, device=DEV), lengths, offsets)
        assert torch.equal(far, near)


@pytest.mark.parametrize("rows", [1, 4, 130])
def test_captured_and_replayed(rows):
    """Two graphs on a workspace each, replayed with other lengths and tables in the same buffers, between eager calls."""
    a = Problem([rows, rows], [700, 300], 2, 4, 128, "affine", 64, "bf16", 16, seed=14)
    eager = a.call()
    T, B, width = a.q.shape[0], 2, a.table.shape[1]
    need = qm.kv_cache_attention_workspace_bytes(a.cache, T, 8, B, width, True)
    ws = [torch.empty(max(need, 16), dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs, graphs = [], []
    for w in ws:
        w.fill_(255)
        out = torch.empty_like(a.q)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            a.call(workspace=w, out=out)
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a.call(workspace=w, out=out)
        outs.append(out)
        graphs.append(graph)
    for lengths in ([700, 300], [rows, 17], [0, 208], [333, 0], [700, 300]):
        a.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
        want = a.call()
        for graph, out in zip(graphs, outs):
            out.fill_(3.0)
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    assert torch.equal(want, eager)


def test_two_streams_at_once():
    ps = [Problem([1] * 8, [3000 + 100 * i] * 8, 2, 4, 128, "affine", 64, "bf16", 64, seed=20 + i) for i in range(2)]
    want = [p.call() for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(10):
        got = []
        for p, s in zip(ps, streams):
            with torch.cuda.stream(s):
                got.append(p.call())
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_refusals():
    p = Problem([2, 2], [40, 40], 2, 2, 64, "affine", 64, "bf16", 16, seed=15)
    args = (p.q, p.cache, p.table, p.lengths)
    for bad in (lambda: qm.kv_cache_attention(p.q.half(), *args[1:], offsets=p.offsets),
                lambda: qm.kv_cache_attention(p.q[:, :, :32], *args[1:], offsets=p.offsets),
                lambda: qm.kv_cache_attention(p.q[0], *args[1:], offsets=p.offsets),
                lambda: qm.kv_cache_attention(p.q, p.cache, p.table[0], p.lengths, offsets=p.offsets),
                lambda: qm.kv_cache_attention(p.q, p.cache, p.table, p.lengths[:1], offsets=p.offsets),
                lambda: qm.kv_cache_attention(*args, offsets=p.offsets[:2]),
                lambda: qm.kv_cache_attention(p.q, p.cache, p.table.long(), p.lengths, offsets=p.offsets),
                lambda: qm.kv_cache_attention(*args, offsets=p.offsets, out=p.q.float())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: qm.kv_cache_attention(*args), lambda: p.call(window=-1), lambda: p.call(scale=float("inf")),
                lambda: qm.kv_cache_attention(p.q[:, :3], *args[1:], offsets=p.offsets)):
        with pytest.raises(qm.QlinError):
            bad()
    long = Problem([1], [5000], 1, 1, 64, "affine", 64, "bf16", 16, seed=16)
    with pytest.raises(qm.QlinError):
        long.call(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    empty = qm.kv_cache_attention(p.q[:0], p.cache, p.table[:0], p.lengths[:0])
    assert empty.shape == (0, 4, 64)
