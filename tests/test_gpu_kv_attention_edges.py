"""Attention over a 4-bit cache on the GPU where blocks of keys hold no values and where keys that no row sees are no
numbers, sequences of 2^30 keys, sizes of values that change. Problems, formulas and tolerances are those of test_gpu_kv_attention."""
import numpy as np
import pytest
import torch

from test_gpu_kv_attention import DEV, DTYPES, Problem, f64

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


@pytest.mark.parametrize("what", ["nan", "large"])
@pytest.mark.parametrize("mode,g", [("affine", 32), ("affine", 64), ("affine", 128), ("mxfp4", 32), ("nvfp4", 16)])
@pytest.mark.parametrize("rows,D,dtype", [(1, 128, "bf16"), (1, 128, "f16"), (5, 64, "bf16"), (40, 128, "bf16"), (300, 128, "bf16"),
                                          (300, 64, "f16"), (1, 256, "bf16"), (3, 160, "f16"), (1, 128, "f32")])
def test_keys_before_the_window_may_be_anything(rows, D, dtype, mode, g, what):
    """What no row sees does not change a bit of the output, be it no number or far larger than what is seen."""
    if D % g:
        pytest.skip("head_dim is no multiple of the group")
    print(f"before the window rows {rows} D{D} {dtype} {mode} g{g} {what}", flush=True)
    window = 45
    p = Problem([rows, rows, rows], [rows + 171, rows + 54, rows + 20], 2, 2 if rows > 1 else 3, D, mode, g, dtype, 16, seed=41,
                garbage=False)
    clean = p.call(window=window)
    p.check(clean, window=window)
    hidden = np.zeros((p.cache.pages, 16), dtype=bool)
    for b, n in enumerate(p.lengths_host):
        for key in range(max(0, n - rows + 1 - window)):
            hidden[p.table_host[b, key // 16], key % 16] = True
    assert hidden.any()
    hole = torch.from_numpy(hidden).to(DEV)[:, None, :, None]
    for w in (p.cache.key, p.cache.value):
        if mode != "affine":
            w.scales.masked_fill_(hole, 255 if what == "nan" else (120 if mode == "nvfp4" else 140))
        else:
            w.scales.masked_fill_(hole, float("nan") if what == "nan" else 4000.0)
            w.biases.masked_fill_(hole, float("inf") if what == "nan" else -3000.0)
    assert torch.equal(p.call(window=window), clean)


@pytest.mark.parametrize("window", [300, 0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sequences_of_2_to_the_30_keys_and_more(dtype, window):
    """One page named again and again: its last places are what a window sees, and every place has the same share of a
    softmax over all of it, however often it comes."""
    page, pages = 1 << 18, 8191 if dtype == "bf16" else 4100
    if dtype == "f32" and not window:
        pytest.skip("the vector units take seconds for these")
    print(f"long {dtype} window {window}", flush=True)
    p = Problem([1], [page], 1, 2, 64, "affine", 64, dtype, page, seed=43, spare=0)
    p.prompt = False
    want, tol = p.want(window=window)
    table = torch.zeros((1, pages), dtype=torch.int32, device=DEV)
    lengths = torch.tensor([pages * page], dtype=torch.int32, device=DEV)
    got = qm.kv_cache_attention(p.q, p.cache, table, lengths, window=window)
    # as many fp32 additions as keys: each sum is off by up to sqrt(keys) of its roundings
    tol = tol + (0 if window else 2 * np.sqrt(pages * page) * 2.0 ** -24 * np.abs(p.dense()[1]).max())
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), (err.max(), tol.min())


@pytest.mark.parametrize("power", [8, 20, 40, 60])
@pytest.mark.parametrize("order", ["down", "up"])
@pytest.mark.parametrize("D,dtype,mode,g", [(64, "bf16", "affine", 64), (128, "bf16", "mxfp4", 32), (192, "bf16", "affine", 32),
                                            (128, "f16", "affine", 64)])
def test_small_values_seen_beside_a_prompts_large_ones(D, dtype, mode, g, order, power):
    """Rows whose window holds small values only, in a prompt whose other values are 2^power times as large, before them or
    behind: what they lose is relative to the blocks of 64 keys that they see (p of 50 keys, each to 2^-21 of the row's largest)."""
    if dtype == "f16" and power > 8:
        pytest.skip("outside f16")
    print(f"sizes {order} 2^{power} D{D} {dtype} {mode}", flush=True)
    rows, window, page = 700, 50, 64
    p = Problem([rows], [rows], 1, 2, D, mode, g, dtype, page, seed=44, garbage=False)
    v = qm.dequantize(p.cache.value, torch.float32) * (1.0 if dtype == "bf16" else 2.0 ** -4)
    # the sequence's middle pages are 2^-power of the others, or the others 2^-power of them
    middle = torch.from_numpy(p.table_host[0, 3:8].astype(np.int64)).to(DEV)
    is_middle = torch.zeros(v.shape[0], dtype=torch.bool, device=DEV)
    is_middle[middle] = True
    small = is_middle if order == "down" else ~is_middle
    v = torch.where(small[:, None, None, None], v * 2.0 ** -power, v)
    p.cache = qm.KVCache(p.cache.key, qm.quantize(v.to(DTYPES[dtype]).contiguous(), g, 4, mode))
    got = p.call(window=window)
    assert qm.last_path() == "kv_attention_prompt"
    p.prompt = True
    want, tol = p.want(window=window)
    values = p.dense()[1]
    tol = tol - 2.0 ** -24 * np.abs(values[p.table_host[0]]).max()       # that of the whole sequence's largest value
    for i in range(rows):
        blocks = np.unique(np.arange(max(0, i - window + 1), i + 1) // page)
        tol[i] += (window * 2.0 ** -21 + 2.0 ** -24) * np.abs(values[p.table_host[0, blocks]]).max()
    err = np.abs(f64(got) - want)
    assert np.isfinite(f64(got)).all()
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("rows", [1, 5, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_the_same_call_gives_the_same_bits(rows, dtype):
    """Between other work, on a workspace that held something else."""
    p = Problem([rows, rows, 1], [5000, 3001, 700], 2, 4, 128, "affine", 64, dtype, 64, seed=42)
    first = p.call()
    need = qm.kv_cache_attention_workspace_bytes(p.cache, p.q.shape[0], 8, 3, p.table.shape[1], True, dtype=DTYPES[dtype])
    for i in range(20):
        ws = torch.full((max(need, 16),), 37 * i % 256, dtype=torch.uint8, device=DEV)
        (torch.randn(1 << 18, device=DEV) * 2.0).sum()
        assert torch.equal(p.call(workspace=ws), first)


@pytest.mark.parametrize("rows", [3, 300])
def test_a_padded_batch_captured_without_an_output(rows):
    """The output and its zeros for rows of no sequence are the graph's own: every replay writes both anew."""
    p = Problem([rows, rows], [400, 350], 2, 2, 128, "affine", 64, "bf16", 32, seed=45)
    q = torch.cat([p.q, torch.full((7, 4, 128), float("nan"), device=DEV, dtype=p.q.dtype)])

    def call():
        return qm.kv_cache_attention(q, p.cache, p.table, p.lengths, offsets=p.offsets)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = call()
    torch.cuda.current_stream().wait_stream(stream)
    for lengths in ([400, 350], [rows, 0], [399, 1], [400, 350]):
        p.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
        want = call()
        (torch.randn(1 << 16, device=DEV) * 2.0).sum()
        out.fill_(5.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and (out[2 * rows :] == 0).all()


@pytest.mark.parametrize("dtype,mode,g", [("f16", "affine", 64), ("bf16", "affine", 64), ("f32", "affine", 64), ("bf16", "mxfp4", 32)])
def test_the_workspace_that_is_asked_for_is_enough(dtype, mode, g):
    """By default for rows of an affine cache's own type."""
    for rows in (1, 300):
        p = Problem([rows], [5000], 2, 2, 64, mode, g, dtype, 64, seed=51)
        need = qm.kv_cache_attention_workspace_bytes(p.cache, rows, 4, 1, p.table.shape[1], True)
        assert (need == 0) == (dtype == "f32")
        got = p.call(workspace=torch.empty(max(need, 16), dtype=torch.uint8, device=DEV))
        assert torch.equal(got, p.call())
