"""Timed cases of the attention operators around a cache of keys and values held in 4 bits: rotary positions (and their
gradient), writing rows into the cache and reading them back, and attention over it.

Plain forms in elementary torch operations stand beside the framework's calls; `exact` states each operator in 64 bits.

The cache is a pool of pages [pages, heads, page, head_dim], quantized along head_dim as the framework quantizes a
weight; a sequence's keys lie in the pages that its row of the page table names.
"""
import math

import torch

own = False

DEVICE = "cuda:0"
FLOATS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]  # magnitudes of a 4-bit float code


def listed():
    return [
        # one token of a decode step: 32 query and 8 key heads, side by side in the row of their projection
        dict(name="rotary_token", op="rotary", T=1, heads=40, tail=8, D=128, R=128, dtype="bf16", interleaved=False,
             factor=1.0, train=False),
        # a training batch of odd length, part of the head rotated, neighbouring pairs, with the gradient
        dict(name="rotary_train", op="rotary", T=8191, heads=20, tail=0, D=96, R=64, dtype="f16", interleaved=True,
             factor=1.0, train=True),
        # a long prompt far behind the trained positions, frequencies scaled for it
        dict(name="rotary_prompt", op="rotary", T=32768, heads=40, tail=8, D=128, R=128, dtype="bf16", interleaved=False,
             factor=8.0, train=False),
        # one decode step of 8 requests: their keys and values go into the cache and are read back
        dict(name="store_step", op="store", T=8, H=8, D=128, dtype="bf16", mode="affine", g=64, page=16, padded=0.0),
        # an odd batch of rows, some of them padding
        dict(name="store_ragged", op="store", T=1027, H=6, D=192, dtype="f16", mode="nvfp4", g=16, page=48, padded=0.1),
        # a long prompt's rows
        dict(name="store_prompt", op="store", T=32768, H=8, D=128, dtype="bf16", mode="affine", g=64, page=64, padded=0.0),
        # the rows of a short prefix, and of a long one, for a product with dense keys
        dict(name="read_prefix", op="read", T=509, H=4, D=256, dtype="bf16", mode="mxfp4", g=32, page=16),
        dict(name="read_long", op="read", T=131072, H=8, D=128, dtype="bf16", mode="affine", g=64, page=128),
        # decode of one short request: latency
        dict(name="attend_token", op="attend", B=1, n=1, L=1500, H=8, G=4, D=128, dtype="bf16", mode="affine", g=64,
             page=16, window=0, causal=True, gaps=False),
        # decode of a large batch with lengths from 8192 to 32768: the cache is what is read
        dict(name="attend_batch", op="attend", B=64, n=1, L=32768, H=8, G=4, D=128, dtype="bf16", mode="affine", g=64,
             page=64, window=0, causal=True, gaps=False),
        # drafted tokens of 16 requests checked at once, behind a window; two requests hold nothing
        dict(name="attend_drafts", op="attend", B=16, n=5, L=20011, H=4, G=7, D=64, dtype="f16", mode="mxfp4", g=32,
             page=32, window=8192, causal=True, gaps=True),
        # a prompt's last 8192 tokens over 16384 keys
        dict(name="attend_prompt", op="attend", B=1, n=8192, L=16384, H=8, G=4, D=128, dtype="bf16", mode="affine", g=64,
             page=64, window=0, causal=True, gaps=False),
    ]


def _log(rng, low, high):
    """A whole number, even over its logarithm; multiples of 96 move one up, as ragged sizes are what a draw is for."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return n + (n % 96 == 0)


def _format(rng, D):
    mode = rng.choice(["affine", "affine", "mxfp4", "nvfp4"])
    return mode, {"mxfp4": 32, "nvfp4": 16}.get(mode) or rng.choice([g for g in (32, 64, 128) if D % g == 0])


def draw(rng):
    op = rng.choice(["rotary", "store", "read", "attend", "attend"])
    if op == "rotary":
        D = rng.choice([64, 80, 96, 128, 192, 256])
        R = rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)])
        heads, tail = rng.randint(1, 48), rng.choice([0, 2, 8])
        train = rng.random() < 0.4
        T = min(_log(rng, 1, 32768), 32768 * 40 * 128 // ((heads + tail) * D * (2 if train else 1)))
        return dict(op=op, T=T, heads=heads, tail=tail, D=D, R=R, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    interleaved=rng.random() < 0.5, factor=rng.choice([1.0, 4.0]), train=train)
    D = rng.choice([64, 96, 128, 128, 192, 256])
    mode, g = _format(rng, D)
    page = 16 * rng.choice([1, 2, 3, 4, 8, 16])
    if op in ("store", "read"):
        H = rng.randint(1, 12)
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        T = _log(rng, 1, 32768 * 8 * 128 // (H * D) // (2 if dtype == "f32" else 1))
        case = dict(op=op, T=T, H=H, D=D, dtype=dtype, mode=mode, g=g, page=page)
        return dict(case, padded=rng.choice([0.0, 0.1])) if op == "store" else case
    dtype = rng.choice(["bf16", "bf16", "f16"])
    H, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8, 16])
    form = rng.choice(["token", "token", "drafts", "prompt"])
    if form == "prompt":
        B, n, L = rng.randint(1, 4), _log(rng, 20, 3000), _log(rng, 30, 8000)
    else:
        B, n, L = _log(rng, 1, 64), 1 if form == "token" else rng.randint(2, 8), _log(rng, 30, 30000)
        B = min(B, max(1, 8_000_000 // (L * H)))
    return dict(op=op, B=B, n=n, L=max(L, n), H=H, G=G, D=D, dtype=dtype, mode=mode, g=g, page=page,
                window=rng.choice([0, 0, rng.randint(1, 4096)]), causal=rng.random() < 0.85, gaps=rng.random() < 0.3)


def _rows_and_lengths(case):
    """Rows of the queries and keys of each sequence, by the case alone. With gaps some sequences hold no keys, and
    some fewer than they have queries, so that rows see nothing."""
    rows, lengths = [], []
    for b in range(case["B"]):
        part = (b * 0.6180339887) % 1.0
        n = case["n"] if b == 0 or case["n"] == 1 else max(1, int(case["n"] * (1 - 0.5 * part)))
        length = max(n, int(case["L"] * (1 - 0.75 * part)))
        if case["gaps"] and b % 8 == 3:
            length = 0
        if case["gaps"] and b % 8 == 6:
            length = n // 2
        rows.append(n)
        lengths.append(length)
    return rows, lengths


def _seen(case, n, length):
    """Pairs of a query and a key it sees, and keys that any query sees, of one sequence."""
    pairs, first = 0, length
    for i in range(n):
        last = length - n + i if case["causal"] else length - 1
        start = max(0, length - n + i - case["window"] + 1) if case["window"] else 0
        start, last = min(start, length), min(last, length - 1)
        if last >= start:
            pairs += last - start + 1
            first = min(first, start)
    return pairs, length - first


# ---------------------------------------------------------------------------------------------------------------- inputs


def _normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEVICE) * std).to(dtype)


def _heads(gen, shape, dtype):
    """Keys or values as projections give them: normal values, a few channels of a head several times larger."""
    wide = torch.where(torch.rand((1,) + shape[1:], generator=gen, device=DEVICE) < 0.03, 4.0, 1.0)
    return ((torch.randn(shape, generator=gen, device=DEVICE) + 0.1) * wide).to(dtype)


def _pool(case, pages, scale_dtype):
    """An empty cache: codes, scales (and biases) of the keys, then of the values."""
    lead = (pages, case["H"], case["page"])
    kind = FLOATS[scale_dtype] if case["mode"] == "affine" else torch.uint8
    out = []
    for _ in range(2):
        out += [torch.zeros(lead + (case["D"] // 8,), dtype=torch.int32, device=DEVICE),
                torch.zeros(lead + (case["D"] // case["g"],), dtype=kind, device=DEVICE),
                torch.zeros(lead + (case["D"] // case["g"],), dtype=kind, device=DEVICE) if case["mode"] == "affine" else None]
    return out


def _handle(case, pool):
    """The framework's handle on a pool."""
    import quantized_matmul_amd as qm

    weights = [qm.QuantizedWeight(*pool[at : at + 3], case["g"], 4, True, case["mode"]) for at in (0, 3)]
    return qm.KVCache(*weights)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    dtype, s = FLOATS[case["dtype"]], {"case": case}
    if case["op"] == "rotary":
        T, D, R = case["T"], case["D"], case["R"]
        rows = _normal(gen, (T, case["heads"] + case["tail"], D), dtype)
        s["x"] = rows[:, : case["heads"]]  # the tail of a projection's row (the values) is not rotated
        start = int(torch.randint(0, 100000, (1,), generator=gen, device=DEVICE))
        s["positions"] = torch.arange(start, start + T, dtype=torch.int32, device=DEVICE)
        turn = torch.arange(0, R, 2, dtype=torch.float64, device=DEVICE) / R
        s["freqs"] = (10000.0**-turn / case["factor"]).float()
        s["grad"] = _normal(gen, (T, case["heads"], D), dtype) if case["train"] else None
        return s
    if case["op"] == "attend":
        rows, lengths = _rows_and_lengths(case)
        page = case["page"]
        need = [-(-n // page) for n in lengths]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32).tolist()
        table = torch.full((case["B"], max(max(need), 1)), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor(order[:n], dtype=torch.int32)
            order = order[n:]
        s["pool"] = _pool(case, pages, case["dtype"])
        for at in (0, 3):  # every page holds rows, those past a sequence's end too
            for p in range(0, pages, 256):
                some = _heads(gen, (min(256, pages - p), case["H"], page, case["D"]), dtype)
                for part, new in zip(s["pool"][at : at + 3], _quantize(case, some)):
                    if part is not None:
                        part[p : p + 256] = new
        s["table"] = table.to(DEVICE)
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=DEVICE)
        starts = [sum(rows[:b]) for b in range(case["B"] + 1)]
        s["offsets"] = torch.tensor(starts, dtype=torch.int32, device=DEVICE) if case["n"] > 1 else None
        s["rows_host"], s["lengths_host"] = rows, lengths  # the plain form's loop
        s["q"] = _normal(gen, (starts[-1], case["H"] * case["G"], case["D"]), dtype, 2.0)
    else:
        T, H, D, page = case["T"], case["H"], case["D"], case["page"]
        pages = -(-T // page) + 2
        places = torch.randperm(pages, generator=gen, device=DEVICE)[:, None] * page + torch.arange(page, device=DEVICE)
        slots = places.reshape(-1)[:T].to(torch.int32)
        s["pool"] = _pool(case, pages, case["dtype"])
        if case["op"] == "store":
            rows = _heads(gen, (T, 6 * H, D), dtype)  # a projection's row: 4 H query heads, then keys, then values
            s["k"], s["v"] = rows[:, 4 * H : 5 * H], rows[:, 5 * H :]
            if case["padded"]:
                slots = torch.where(torch.rand(T, generator=gen, device=DEVICE) < case["padded"], -1, slots)
        else:
            for at in (0, 3):
                for part, new in zip(s["pool"][at : at + 3], _quantize(case, _heads(gen, (pages, H, page, D), dtype))):
                    if part is not None:
                        part.copy_(new)
        s["slots"] = slots.to(torch.int32).contiguous()
    if own:
        s["cache"] = _handle(case, s["pool"])
    return s


# ----------------------------------------------------------------------------------------------------------- plain forms


def _directed(v, dtype, up):
    """v in 32 bits rounded to dtype towards +infinity or -infinity."""
    if dtype == torch.float32:
        return v
    h = v.to(dtype)
    wrong = h.float() < v if up else h.float() > v
    bits = h.view(torch.int16)
    away = (bits >= 0) == up  # one step up of a positive number, or down of a negative one, grows its pattern
    moved = torch.where(h == 0, torch.full_like(bits, 1 if up else -32767), torch.where(away, bits + 1, bits - 1))
    return torch.where(wrong, moved, bits).view(dtype).float()


def _quotient(a, b):
    """a / b of 32-bit numbers, rounded once (a division by a plain number may be a product with its reciprocal)."""
    return (a.double() / (b if torch.is_tensor(b) else torch.full_like(a, b))).float()


def _pack(codes):
    shift = torch.arange(0, 32, 4, device=codes.device, dtype=torch.int32)
    return (codes.reshape(codes.shape[:-1] + (-1, 8)) << shift).sum(-1, dtype=torch.int32)


def _two(e):
    """2^e of whole numbers e in [-127, 127], in 32 bits, from its pattern."""
    e = e.int()
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).int().view(torch.float32)


def _nearest_code(v):
    """Code of the nearest 4-bit float, a tie to the even code."""
    a = v.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())
    return code + 8 * torch.signbit(v).int()


def _quantize(case, x):
    """(codes, scales, biases) of x along its last axis in the cache's format."""
    mode, g = case["mode"], case["g"]
    v = x.float().reshape(x.shape[:-1] + (-1, g))
    if mode == "affine":
        z = _directed(v.amin(-1, keepdim=True), x.dtype, False)
        s = _directed(_quotient(v.amax(-1, keepdim=True) - z, 15.0), x.dtype, True)
        q = torch.where(s > 0, torch.round(_quotient(v - z, torch.where(s > 0, s, 1.0))), 0.0).clamp(0, 15)
        return _pack(q.int().reshape(x.shape)), s.squeeze(-1).to(x.dtype), z.squeeze(-1).to(x.dtype)
    most = v.abs().amax(-1, keepdim=True)
    if mode == "mxfp4":
        e = torch.where(most > 0, torch.frexp(most)[1] - 3, torch.full_like(most, -127, dtype=torch.int32)).clamp(-127, 127)
        code = _nearest_code(v * _two(-(e // 2)) * _two(-(e - e // 2)))
        return _pack(code.reshape(x.shape)), (e + 127).squeeze(-1).to(torch.uint8), None
    byte = _quotient(most, 6.0).to(torch.float8_e4m3fn)
    s = byte.float()
    code = _nearest_code(torch.where(s > 0, _quotient(v, torch.where(s > 0, s, 1.0)), 0.0))
    return _pack(code.reshape(x.shape)), byte.view(torch.uint8).squeeze(-1), None


def _values(case, words, scales, biases):
    """The numbers, in 32 bits, that codes with their scales (and biases) stand for."""
    shift = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    codes = ((words[..., None] >> shift) & 15).reshape(scales.shape + (case["g"],))
    if case["mode"] == "affine":
        v = scales.float()[..., None] * codes + biases.float()[..., None]
    else:
        v = torch.tensor(LEVELS + [-a for a in LEVELS], device=words.device)[codes]
        if case["mode"] == "mxfp4":
            v = v * _two(scales.int() - 127)[..., None]
        else:
            v = v * scales.view(torch.float8_e4m3fn).float()[..., None]
    return v.reshape(words.shape[:-1] + (-1,))


def _plain_rotary(case, s):
    R, half = case["R"], case["R"] // 2
    angle = s["positions"].double()[:, None] * s["freqs"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turned(x, sin):
        out = x.float()
        a, b = (out[..., 0:R:2], out[..., 1:R:2]) if case["interleaved"] else (out[..., :half], out[..., half:R])
        pair = a * cos - b * sin, a * sin + b * cos
        mixed = torch.stack(pair, -1).flatten(-2) if case["interleaved"] else torch.cat(pair, -1)
        return torch.cat([mixed, out[..., R:]], -1).to(x.dtype)

    return [turned(s["x"], sin)] + ([turned(s["grad"], -sin)] if case["train"] else [])


def _plain_read(case, pool, slots):
    page, live = case["page"], slots >= 0
    at = slots.clamp_min(0).long()
    p, o = at // page, at % page
    out = []
    for k in (0, 3):
        v = _values(case, *[None if t is None else t[p, :, o] for t in pool[k : k + 3]])
        out.append(torch.where(live[:, None, None], v, 0.0).to(FLOATS[case["dtype"]]))
    return out


def _plain_store(case, s):
    at = s["slots"][s["slots"] >= 0].long()
    p, o = at // case["page"], at % case["page"]
    for k, x in ((0, s["k"]), (3, s["v"])):
        for part, new in zip(s["pool"][k : k + 3], _quantize(case, x[s["slots"] >= 0])):
            if part is not None:
                part[p, :, o] = new
    return _plain_read(case, s["pool"], s["slots"])


def _plain_attend(case, s):
    H, G, D, page = case["H"], case["G"], case["D"], case["page"]
    out, first = torch.zeros_like(s["q"]), 0
    for b, (n, length) in enumerate(zip(s["rows_host"], s["lengths_host"])):
        if length:
            pages = s["table"][b, : -(-length // page)].long()
            k, v = [_values(case, *[None if t is None else t[pages].transpose(1, 2) for t in s["pool"][at : at + 3]])
                    .reshape(-1, H, D)[:length].transpose(0, 1) for at in (0, 3)]
            step = max(1, (1 << 30) // (H * G * length))
            for i in range(0, n, step):
                rows = s["q"][first + i : first + min(n, i + step)].float()
                m = rows.shape[0]
                rows = rows.view(m, H, G, D).transpose(0, 1).reshape(H, m * G, D)
                score = torch.matmul(rows, k.transpose(1, 2)).view(H, m, G, length) * D**-0.5
                at = length - n + i + torch.arange(m, device=score.device)[:, None]
                key = torch.arange(length, device=score.device)[None]
                seen = key <= at if case["causal"] else key >= 0
                if case["window"]:
                    seen = seen & (key > at - case["window"])
                score = torch.where(seen[None, :, None], score, -math.inf)
                top = score.amax(-1, keepdim=True).clamp_min(-1e30)
                p = torch.exp(score - top)
                p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
                o = torch.matmul(p.view(H, m * G, length), v).view(H, m, G, D).transpose(0, 1)
                out[first + i : first + i + m] = o.reshape(m, H * G, D).to(out.dtype)
        first += n
    return [out]


def _plain(case, s):
    if case["op"] == "rotary":
        return _plain_rotary(case, s)
    if case["op"] == "store":
        return _plain_store(case, s)
    return _plain_read(case, s["pool"], s["slots"]) if case["op"] == "read" else _plain_attend(case, s)


# ------------------------------------------------------------------------------------------------- the framework's calls


def _framework(case, s):
    import quantized_matmul_amd as qm

    if case["op"] == "rotary":
        out = [qm.rotary(s["x"], s["positions"], s["freqs"], interleaved=case["interleaved"])]
        if case["train"]:
            out.append(qm.rotary_grad(s["grad"], s["positions"], s["freqs"], interleaved=case["interleaved"]))
        return out
    if case["op"] == "attend":
        return [qm.kv_cache_attention(s["q"], s["cache"], s["table"], s["lengths"], offsets=s["offsets"],
                                      causal=case["causal"], window=case["window"])]
    if case["op"] == "store":
        qm.kv_cache_write(s["cache"], s["k"], s["v"], s["slots"])
    return list(qm.kv_cache_read(s["cache"], s["slots"], dtype=FLOATS[case["dtype"]]))


def run(state):
    return (_framework if own else _plain)(state["case"], state)


def work(case):
    size, D = SIZE[case["dtype"]], case["D"]
    if case["op"] == "rotary":
        x = case["T"] * case["heads"] * D * (2 if case["train"] else 1)
        return {"bytes": 2 * x * size + case["T"] * 4 + case["R"] * 2, "flops": 3 * x}
    held = D // 2 + D // case["g"] * (2 * size if case["mode"] == "affine" else 1)  # bytes of a head's row
    if case["op"] == "attend":
        q, pairs, keys = 0, 0, 0
        for n, length in zip(*_rows_and_lengths(case)):
            a, b = _seen(case, n, length)
            q, pairs, keys = q + n, pairs + a, keys + b
        return {"bytes": 2 * q * case["H"] * case["G"] * D * size + 2 * keys * case["H"] * held,
                "flops": 4 * pairs * case["H"] * case["G"] * D}
    rows = 2 * case["T"] * case["H"]
    if case["op"] == "read":
        return {"bytes": rows * (held + D * size) + 4 * case["T"], "flops": 2 * rows * D}
    return {"bytes": rows * (2 * held + 2 * D * size) + 8 * case["T"], "flops": 8 * rows * D}


# --------------------------------------------------------------------------------------------------------- 64-bit values


def _power(e):
    """2^e of whole numbers e, in 64 bits, from its pattern."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(case, words, scales, biases):
    out = []
    for place in range(8):
        code = (words.long() >> (4 * place)) & 15
        if case["mode"] == "affine":
            out.append(code.double())
            continue
        power, half = (code >> 1) & 3, (code & 1).double()
        size = torch.where(power > 0, (1 + half / 2) * _power(power - 1), half / 2)
        out.append(torch.where(code >= 8, -size, size))
    v = torch.stack(out, -1).reshape(scales.shape + (case["g"],))
    if case["mode"] == "affine":
        v = v * scales.double()[..., None] + biases.double()[..., None]
    elif case["mode"] == "mxfp4":
        v = v * _power(scales.long() - 127)[..., None]
    else:
        e, m = (scales.long() >> 3) & 15, (scales.long() & 7).double()
        v = v * torch.where(e > 0, (1 + m / 8) * _power(e - 7), m / 8 * 2.0**-6)[..., None]
    return v.reshape(words.shape[:-1] + (-1,))


def _grid(v, dtype):
    """Distance of dtype's numbers around v, in 64 bits."""
    bits, low = (8, -133) if dtype == torch.bfloat16 else (11, -24)
    return _power((torch.frexp(v)[1] - bits).clamp_min(low))


def _exact_rounded(case, x):
    """The numbers that x is held as. Scale, bias and quotient are defined with the roundings of 32 bits."""
    v = x.float().double().reshape(x.shape[:-1] + (-1, case["g"]))
    low, high = v.min(-1, keepdim=True)[0], v.max(-1, keepdim=True)[0]
    if case["mode"] == "affine":
        s = ((high - low).float().double() / torch.full_like(high, 15.0)).float().double()  # the group's lowest value is one of x's own
        if x.dtype != torch.float32:
            step = _grid(s, x.dtype)
            s = torch.ceil(s / step) * step
        q = ((v - low).float().double() / torch.where(s > 0, s, 1.0)).float().double().round().clamp(0, 15)
        out = torch.where(s > 0, q * s, 0.0) + low
    else:
        most = torch.maximum(high, -low)
        if case["mode"] == "mxfp4":
            unit = _power((torch.frexp(most)[1] - 3).clamp(-127, 127))
        else:
            t = (most / torch.full_like(most, 6.0)).float().double()
            step = _power((torch.frexp(t)[1] - 4).clamp_min(-9))
            unit = ((t / step).round() * step).clamp_max(448.0)
        t = (v / torch.where(unit > 0, unit, 1.0)).float().double()
        a = t.abs().clamp_max(6.0)
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
        out = torch.where(unit > 0, torch.sign(t) * (a / step).round() * step * unit, 0.0)  # ties to even: the even code
    return out.reshape(x.shape)


def _exact_attend(case, s):
    H, G, D, page = case["H"], case["G"], case["D"], case["page"]
    out, first = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE), 0
    for b, (n, length) in enumerate(zip(*_rows_and_lengths(case))):
        key = torch.arange(length, device=DEVICE)
        page_of, place = s["table"][b].long()[key // page], key % page
        for h in range(H if length else 0):
            k, v = [_exact_values(case, *[None if t is None else t[page_of, h, place] for t in s["pool"][at : at + 3]])
                    for at in (0, 3)]
            k = k.t().contiguous()
            step = max(1, (1 << 28) // (G * length))
            for i in range(0, n, step):
                m = min(step, n - i)
                q = s["q"][first + i : first + i + m, h * G : (h + 1) * G].double().reshape(m * G, D)
                at = (length - n + i + torch.arange(m, device=DEVICE)).repeat_interleave(G)[:, None]
                hidden = torch.zeros((m * G, length), dtype=torch.bool, device=DEVICE)
                if case["causal"]:
                    hidden |= key[None] > at
                if case["window"]:
                    hidden |= key[None] <= at - case["window"]
                p = torch.softmax((q @ k / math.sqrt(D)).masked_fill(hidden, -math.inf), -1)
                o = torch.nan_to_num(p) @ v
                out[first + i : first + i + m, h * G : (h + 1) * G] = o.view(m, G, D)
        first += n
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return [_exact_attend(case, s)]
    if case["op"] == "rotary":
        R = case["R"]
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEVICE),
                           s["positions"].double()[:, None] * s["freqs"].double())[:, None]
        out = []
        for x, by in ((s["x"], turn), (s["grad"], turn.conj())):
            if x is None:
                continue
            y = x.double().clone()
            first, second = (slice(0, R, 2), slice(1, R, 2)) if case["interleaved"] else (slice(0, R // 2), slice(R // 2, R))
            z = torch.complex(y[..., first], y[..., second]) * by
            y[..., first], y[..., second] = z.real, z.imag
            out.append(y)
        return out
    live = (s["slots"] >= 0)[:, None, None]
    if case["op"] == "store":
        return [torch.where(live, _exact_rounded(case, x), 0.0) for x in (s["k"], s["v"])]
    at = s["slots"].long()
    p, o = at // case["page"], at % case["page"]
    return [_exact_values(case, *[None if t is None else t[p, :, o] for t in s["pool"][k : k + 3]]) for k in (0, 3)]
