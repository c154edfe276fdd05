"""An attention layer on quantized weights and a 4-bit cache of keys and values, serving prompts and single tokens.

A step, for the rows x [T, D] of any number of requests (HQ query heads and H key heads of width d):
    qkv   = quantized_matmul(x, w_in)              [T, (HQ + 2 H) d]
    q, k  = rotary(q, k)                           in place, the values of a row stay
    kv_cache_write(k, v) at the rows' slots
    o     = kv_cache_attention(q)                  [T, HQ d], over each request's pages
    y     = quantized_matmul(o, w_out)             [T, D]
Nothing in it asks the GPU for a number, so a step of single tokens is captured
once into a graph and replayed for each token.

    python examples/attention_layer.py [--requests 16] [--prompt 1024] [--tokens 64] [--dim 4096] [--heads 32]
                                       [--key-heads 8] [--mode affine]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_matmul_amd as qm  # noqa: E402


class AttentionLayer:
    """w_in [(HQ + 2 H) d, D] and w_out [D, HQ d], quantized here to 4 bits in groups of 64."""

    def __init__(self, w_in, w_out, heads, key_heads, freqs):
        self.w_in, self.w_out = qm.quantize(w_in, 64, 4), qm.quantize(w_out, 64, 4)
        self.heads, self.key_heads = heads, key_heads
        self.dim = w_in.shape[0] // (heads + 2 * key_heads)
        self.freqs = freqs

    def forward(self, x, cache, positions, slots, table, lengths, offsets=None, window=0):
        """y [T, D]; positions and slots are the rows', table, lengths and offsets the requests' with those rows in."""
        q, k, v = self.project(x, positions)
        qm.kv_cache_write(cache, k, v, slots)
        o = qm.kv_cache_attention(q, cache, table, lengths, offsets, window=window)
        return qm.quantized_matmul(o.view(x.shape[0], -1), self.w_out)

    def project(self, x, positions):
        """q, k and v of x, turned by their positions."""
        HQ, H = self.heads, self.key_heads
        qkv = qm.quantized_matmul(x, self.w_in).view(x.shape[0], HQ + 2 * H, self.dim)
        turned = qkv[:, : HQ + H]
        qm.rotary(turned, positions, self.freqs, out=turned)
        return qkv[:, :HQ], qkv[:, HQ : HQ + H], qkv[:, HQ + H :]


class Requests:
    """Which pages of a cache each of B requests has, and how many tokens are in them."""

    def __init__(self, B, most, page, device="cuda", seed=0):
        self.page = page
        width = -(-most // page)
        order = torch.randperm(B * width, generator=torch.Generator().manual_seed(seed))
        self.table_host = order.view(B, width).to(torch.int32)
        self.lengths_host = [0] * B
        self.table = self.table_host.to(device)
        self.pages = B * width

    def add(self, counts):
        """Room for counts[b] more tokens of each request: their positions and slots, the requests' new lengths and
        offsets, on the host."""
        positions, slots, offsets = [], [], [0]
        for b, n in enumerate(counts):
            at = torch.arange(self.lengths_host[b], self.lengths_host[b] + n)
            positions.append(at)
            slots.append(self.table_host[b, at // self.page] * self.page + at % self.page)
            self.lengths_host[b] += n
            offsets.append(offsets[-1] + n)
        return [torch.cat(positions).int(), torch.cat(slots).int(), torch.tensor(self.lengths_host, dtype=torch.int32),
                torch.tensor(offsets, dtype=torch.int32)]


class TokenStep:
    """A step of one token of each request, captured into a graph over buffers of its own."""

    def __init__(self, layer, cache, requests):
        B, D = requests.table.shape[0], layer.w_out.shape[0]
        device = requests.table.device
        self.x = torch.zeros(B, D, dtype=torch.bfloat16, device=device)
        self.positions = torch.zeros(B, dtype=torch.int32, device=device)
        self.slots = torch.full((B,), -1, dtype=torch.int32, device=device)     # the pass before capturing writes no row
        self.lengths = torch.zeros(B, dtype=torch.int32, device=device)

        def step():
            return layer.forward(self.x, cache, self.positions, self.slots, requests.table, self.lengths)

        stream = torch.cuda.Stream(device)
        stream.wait_stream(torch.cuda.current_stream(device))
        with torch.cuda.stream(stream):
            step()
        torch.cuda.current_stream(device).wait_stream(stream)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = step()

    def __call__(self, x, positions, slots, lengths):
        """y of the token rows x; the next call writes over it."""
        for buffer, value in ((self.x, x), (self.positions, positions), (self.slots, slots), (self.lengths, lengths)):
            buffer.copy_(value)
        self.graph.replay()
        return self.y


def random_layer(D, heads, key_heads, dim, device="cuda", seed=0):
    g = torch.Generator(device).manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(*shape, generator=g, device=device) * std).bfloat16()

    return AttentionLayer(normal((heads + 2 * key_heads) * dim, D, std=D ** -0.5),
                          normal(D, heads * dim, std=(heads * dim) ** -0.5), heads, key_heads,
                          qm.rotary_frequencies(dim, device=device))


def serve(layer, B, prompt, tokens, mode="affine", page=64, seed=1):
    """Prompts of B requests at once, then `tokens` single tokens of each; returns the outputs of the last step and the
    milliseconds of the prompts and of a token step."""
    device = layer.freqs.device
    requests = Requests(B, prompt + tokens, page, device)
    cache = qm.kv_cache(requests.pages, layer.key_heads, page, layer.dim, mode=mode, device=device)
    g = torch.Generator(device).manual_seed(seed)

    def rows(n):
        return torch.randn(n, layer.w_out.shape[0], generator=g, device=device).bfloat16()

    marks = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    x, where = rows(B * prompt), [t.to(device) for t in requests.add([prompt] * B)]
    step = TokenStep(layer, cache, requests)
    marks[0].record()
    y = layer.forward(x, cache, where[0], where[1], requests.table, where[2], where[3])
    marks[1].record()
    for _ in range(tokens):
        positions, slots, lengths, _ = requests.add([1] * B)
        y = step(rows(B), positions, slots, lengths)
    marks[2].record()
    torch.cuda.synchronize()
    return y, marks[0].elapsed_time(marks[1]), marks[1].elapsed_time(marks[2]) / max(tokens, 1)


def main(argv=None):
    p = argparse.ArgumentParser(description="An attention layer on quantized weights and a 4-bit cache.")
    for name, value in (("requests", 16), ("prompt", 1024), ("tokens", 64), ("dim", 4096), ("heads", 32), ("key-heads", 8)):
        p.add_argument("--" + name, type=int, default=value)
    p.add_argument("--mode", default="affine", choices=("affine", "mxfp4", "nvfp4"))
    a = p.parse_args(argv)
    layer = random_layer(a.dim, a.heads, a.key_heads, 128)
    serve(layer, a.requests, min(a.prompt, 64), 2, a.mode)
    y, prompts, token = serve(layer, a.requests, a.prompt, a.tokens, a.mode)
    print(f"prompts of {a.requests} x {a.prompt} tokens: {prompts:.2f} ms", flush=True)
    print(f"a token of each of {a.requests} requests: {token * 1e3:.1f} us", flush=True)
    return y


if __name__ == "__main__":
    main()
