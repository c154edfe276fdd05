"""Timed cases of the mixture-of-experts operators: routing tokens to experts, products of two mxfp4 operands (dense and
by experts) and the weighted combine of the experts' rows, with the gradients of routing and combining.

Plain forms in elementary torch operations stand beside the framework's calls; `exact` states each operator in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda:0"
FLOATS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
GROUP = 32  # values along K that share one scale in mxfp4


def listed():
    return [
        # one token of a decode step picks 8 of 64 experts: a call that is all latency
        dict(name="route_token", op="route", T=1, E=64, k=8, dtype="bf16", score="softmax", bias=False, groups=1,
             kept=1, top=1, renorm=True, scale=1.0, train=False, dead=0.0),
        # a long prompt batch with a balance bias: the 4 best of 8 groups, then 8 of the 256 experts in them
        dict(name="route_groups", op="route", T=16384, E=256, k=8, dtype="f32", score="sigmoid", bias=True, groups=8,
             kept=4, top=2, renorm=True, scale=2.5, train=False, dead=0.0),
        # a training batch of odd length and an odd number of experts: choice and the gradient of the logits
        dict(name="route_train", op="route", T=8191, E=60, k=4, dtype="bf16", score="softmax", bias=False, groups=1,
             kept=1, top=1, renorm=False, scale=1.0, train=True, dead=0.02),
        # decode with one row against the framework's decode weight [14336, 4096]
        dict(name="dense_row", op="dense", M=1, N=14336, K=4096, dtype="bf16", swiglu=False),
        # a ragged batch of rows against the microscaled weight [8192, 8192], through the gated activation
        dict(name="dense_ragged", op="dense", M=497, N=8192, K=8192, dtype="f16", swiglu=True),
        # a long prompt against the prefill weight [12288, 4096]
        dict(name="dense_prompt", op="dense", M=8192, N=12288, K=4096, dtype="bf16", swiglu=False),
        # one decode token through its 8 of 64 experts
        dict(name="experts_token", op="experts", T=1, k=8, E=64, N=1536, K=2048, dtype="bf16", swiglu=False, dropped=0.0),
        # 512 tokens through 8 of 64 experts, the framework's expert workload, some places dropped
        dict(name="experts_batch", op="experts", T=512, k=8, E=64, N=1536, K=2048, dtype="bf16", swiglu=False, dropped=0.03),
        # 8192 tokens' gate and up rows (one entry per token and place) through the experts' second products
        dict(name="experts_prompt", op="experts", T=65536, k=1, E=64, N=4096, K=2048, dtype="bf16", swiglu=True, dropped=0.0),
        # one decode token's 8 expert rows joined
        dict(name="combine_token", op="combine", T=1, k=8, D=2048, dtype="bf16", train=False, dropped=0.0),
        # an odd batch with dropped places
        dict(name="combine_ragged", op="combine", T=515, k=6, D=2568, dtype="f16", train=False, dropped=0.05),
        # a training batch: the joined rows, and the gradients of rows and weights
        dict(name="combine_train", op="combine", T=8192, k=8, D=4096, dtype="bf16", train=True, dropped=0.0),
    ]


def _log(rng, low, high):
    """A whole number, even over its logarithm; multiples of 96 move one up, as ragged sizes are what a draw is for."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return n + (n % 96 == 0)


def draw(rng):
    op = rng.choice(["route", "dense", "experts", "combine"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "route":
        score = rng.choice(["softmax", "sigmoid"])
        E, groups, kept, top = rng.randint(4, 300), 1, 1, 1
        if rng.random() < 0.4:
            groups = rng.choice([2, 4, 8])
            E, kept, top = groups * rng.randint(8, 32), rng.randint(1, groups), rng.choice([1, 2])
        k = rng.randint(1, min(8, kept * (E // groups)))
        T = min(_log(rng, 1, 16384), 16384 * 256 // E)
        return dict(op=op, T=T, E=E, k=k, dtype=dtype, score=score, bias=rng.random() < 0.5, groups=groups, kept=kept,
                    top=top, renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), train=rng.random() < 0.4,
                    dead=rng.choice([0.0, 0.02]))
    if op == "dense":
        N, K = _log(rng, 200, 14336), GROUP * _log(rng, 8, 256)
        return dict(op=op, M=_log(rng, 1, 8192), N=N, K=K, dtype=dtype, swiglu=rng.random() < 0.3)
    if op == "experts":
        E, N, K = rng.randint(4, 96), _log(rng, 256, 4096), GROUP * _log(rng, 8, 64)
        k = rng.randint(1, min(8, E))
        return dict(op=op, T=_log(rng, 1, 32768 // k), k=k, E=E, N=N, K=K, dtype=dtype, swiglu=rng.random() < 0.3,
                    dropped=rng.choice([0.0, 0.05]))
    return dict(op=op, T=_log(rng, 1, 8192), k=rng.randint(1, 8), D=8 * _log(rng, 16, 512) + rng.choice([0, 0, 1, 4]),
                dtype=dtype, train=rng.random() < 0.5, dropped=rng.choice([0.0, 0.05]))


# ---------------------------------------------------------------------------------------------------------------- inputs


def _normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEVICE) * std).to(dtype)


def _keep_clear(case, logits, bias):
    """Tokens whose choice hangs on the last bits of a 32-bit sum get the next clear token's logits, so that a choice is
    right or wrong and never a matter of rounding. Equal logits stay as they are: those ties have an answer."""
    if not case["bias"] and case["groups"] == 1:
        return logits
    T, E, G = case["T"], case["E"], case["groups"]
    x = logits.double()
    s = torch.softmax(x, 1) if case["score"] == "softmax" else torch.sigmoid(x)
    key = s + bias.double() if case["bias"] else s
    ordered = torch.sort(key.view(T, G, E // G), dim=2, descending=True)[0]
    near = torch.zeros(T, dtype=torch.bool, device=x.device)
    if G > 1 and case["kept"] < G:
        group = ordered[:, :, : case["top"]].sum(2) if E // G > 1 else ordered[:, :, 0]
        g = torch.sort(group, dim=1, descending=True)[0]
        near |= g[:, case["kept"] - 1] - g[:, case["kept"]] < 4e-6
        cut = g[:, case["kept"] - 1]
        key = key.view(T, G, E // G).masked_fill((group < cut[:, None])[:, :, None], -math.inf).view(T, E)
    top = torch.sort(key, dim=1, descending=True)[0][:, : case["k"] + 1]
    gaps = top[:, :-1] - top[:, 1:]
    if case["bias"]:
        near |= (gaps < 4e-6).any(1)
    clear = torch.nonzero(~near)[:, 0]
    at = torch.searchsorted(clear, torch.arange(T, device=x.device)) % clear.numel()
    return logits[clear[at]].contiguous()


def _choices(gen, T, k, E, dropped):
    """k distinct experts for each token, some experts more in demand than others; -1 where a place is dropped."""
    demand = torch.randn((1, E), generator=gen, device=DEVICE) * 0.5
    order = torch.argsort(torch.randn((T, E), generator=gen, device=DEVICE) + demand, dim=1, descending=True)[:, :k]
    ids = order.to(torch.int32)
    if dropped:
        ids = torch.where(torch.rand((T, k), generator=gen, device=DEVICE) < dropped, -torch.ones_like(ids), ids)
    return ids.contiguous()


def _weight(gen, shape):
    """A weight in mxfp4 as a model keeps it: packed codes and scale bytes of normal values."""
    codes, scales = zip(*[_quantize(torch.randn((1,) + shape[1:], generator=gen, device=DEVICE) * 0.02)
                          for _ in range(shape[0])])
    return torch.cat(codes), torch.cat(scales)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    dtype, s = FLOATS[case.get("dtype", "bf16")], {"case": case}
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        bias = torch.randn(E, generator=gen, device=DEVICE) * 0.05 if case["bias"] else None
        logits = _normal(gen, (T + 64, E), dtype, 1.5)  # spare tokens for _keep_clear
        logits = _keep_clear(dict(case, T=T + 64), logits, bias)[:T].contiguous()
        if case["dead"]:
            rare = torch.rand((T, E), generator=gen, device=DEVICE) < case["dead"]
            if not case["bias"] and case["groups"] == 1:  # experts masked for a token; one token without any expert
                logits = logits.masked_fill(rare, -math.inf)
                logits[T // 2] = -math.inf
        s.update(logits=logits, bias=bias)
        s["grad"] = torch.randn((T, case["k"]), generator=gen, device=DEVICE) if case["train"] else None
    elif case["op"] == "dense":
        s["w"], s["ws"] = (t[0].contiguous() for t in _weight(gen, (1, case["N"], case["K"])))
        s["x"] = _normal(gen, (case["M"], case["K"] * (2 if case["swiglu"] else 1)), dtype)
    elif case["op"] == "experts":
        s["w"], s["ws"] = _weight(gen, (case["E"], case["N"], case["K"]))
        s["x"] = _normal(gen, (case["T"], case["K"] * (2 if case["swiglu"] else 1)), dtype)
        s["ids"] = _choices(gen, case["T"], case["k"], case["E"], case["dropped"])
        ids = s["ids"].reshape(-1)
        s["most"] = int(torch.bincount(ids[ids >= 0].long(), minlength=1).max())  # rows of the busiest expert
    else:
        T, k, D = case["T"], case["k"], case["D"]
        s["h"] = _normal(gen, (T, k, D), dtype)
        s["weights"] = torch.softmax(torch.randn((T, k), generator=gen, device=DEVICE), 1)
        s["ids"] = _choices(gen, T, k, max(8, k), case["dropped"]) if case["dropped"] else None
        s["gy"] = _normal(gen, (T, D), dtype) if case["train"] else None
    return s


# ----------------------------------------------------------------------------------------------------------- plain forms


def _quantize(x):
    """mxfp4 of x along its last axis: int32 words of eight E2M1 codes, lowest first, and E8M0 scale bytes."""
    x = x.float()
    blocks = x.reshape(x.shape[:-1] + (-1, GROUP))
    most = blocks.abs().amax(-1, keepdim=True)
    e = torch.where(most > 0, torch.frexp(most)[1] - 3, torch.full_like(most, -127, dtype=torch.int32)).clamp(-127, 127)
    v = torch.ldexp(torch.ldexp(blocks, -(e // 2)), -(e - e // 2))
    a = v.abs()
    # nearest of 0 .5 1 1.5 2 3 4 6, a tie to the even code
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())
    code = (code + 8 * torch.signbit(v).int()).reshape(x.shape[:-1] + (-1, 8))
    shift = torch.arange(0, 32, 4, device=x.device, dtype=torch.int32)
    words = (code << shift).sum(-1, dtype=torch.int32)
    return words, (e + 127).squeeze(-1).to(torch.uint8)


def _values(words, scales):
    """The numbers that mxfp4 words and scale bytes stand for."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=words.device)
    shift = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    codes = (words[..., None] >> shift) & 15
    v = table[codes.reshape(words.shape[:-1] + (-1, GROUP))]
    return torch.ldexp(v, scales.to(torch.int32)[..., None] - 127).reshape(words.shape[:-1] + (-1,))


def _activation(x, swiglu):
    x = x.float()
    if swiglu:
        gate, up = x.chunk(2, -1)
        x = gate / (1 + torch.exp(-gate)) * up
    return _values(*_quantize(x))


def _scores(x, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    return e / e.sum(1, keepdim=True).clamp_min(1e-30)


def _plain_route(case, s):
    T, E, G, k = case["T"], case["E"], case["groups"], case["k"]
    x = s["logits"].float()
    score = _scores(x, case["score"])
    free = torch.isfinite(x)
    value = score + s["bias"] if case["bias"] else score
    key = torch.where(free, value if case["bias"] else x, -math.inf)
    if case["kept"] < G:
        inner = torch.where(free, value, -math.inf).view(T, G, E // G)
        best = torch.sort(inner, dim=2, descending=True, stable=True)[0][:, :, : case["top"]].sum(2)
        rank = torch.sort(best, dim=1, descending=True, stable=True)[1][:, : case["kept"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=x.device).scatter_(1, rank, True)
        key = torch.where(keep[:, :, None], key.view(T, G, E // G), -math.inf).view(T, E)
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    taken = top > -math.inf
    chosen = torch.where(taken, score.gather(1, ids), 0.0)
    total = chosen.sum(1, keepdim=True) + 1e-20 if case["renorm"] else 1.0
    weights = case["scale"] * chosen / total
    out = [weights, torch.where(taken, ids, -1).to(torch.int32)]
    if case["train"]:
        g = torch.where(taken, s["grad"], 0.0)
        c = case["scale"]
        d = (c * g - (g * weights).sum(1, keepdim=True)) / total if case["renorm"] else c * g
        if case["score"] == "sigmoid":
            part = d * chosen * (1 / (1 + torch.exp(x.gather(1, ids))))
            gx = torch.zeros_like(x).scatter_(1, ids, torch.where(taken, part, 0.0))
        elif case["renorm"]:
            gx = torch.zeros_like(x).scatter_(1, ids, torch.where(taken, chosen * d, 0.0))
        else:
            spread = torch.zeros_like(x).scatter_(1, ids, torch.where(taken, d, 0.0))
            gx = score * (spread - (d * chosen).sum(1, keepdim=True))
        out.append(gx.to(s["logits"].dtype))
    return out


def _plain_experts(case, s):
    E, k, N = case["E"], case["k"], case["N"]
    x, ids = _activation(s["x"], case["swiglu"]), s["ids"].reshape(-1).long()
    R = ids.numel()
    live = ids >= 0
    rows = x.repeat_interleave(k, 0)
    if R <= E:  # fewer rows than experts: each row with a copy of its expert
        picked = ids.clamp_min(0)
        y = (_values(s["w"][picked], s["ws"][picked]) * rows[:, None, :]).sum(2)
    else:  # rows laid out by expert, as many places for each as the busiest has
        slot = torch.where(live, ids, E)
        order = torch.argsort(slot, stable=True)
        count = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, slot, torch.ones_like(slot))
        first = torch.cumsum(count, 0) - count
        place = torch.empty_like(order).scatter_(0, order, torch.arange(R, device=ids.device)) - first[slot]
        at = torch.where(live, ids * s["most"] + place, E * s["most"])
        padded = rows.new_zeros((E * s["most"] + 1, rows.shape[1])).index_copy_(0, at[live], rows[live])
        y = torch.matmul(padded[:-1].view(E, s["most"], -1), _values(s["w"], s["ws"]).transpose(1, 2))
        y = y.reshape(E * s["most"], N)[at.clamp_max(E * s["most"] - 1)]
    y = torch.where(live[:, None], y, 0.0)
    return [y.to(s["x"].dtype).view(case["T"], k, N)]


def _plain_combine(case, s):
    h, w = s["h"].float(), s["weights"]
    live = s["ids"] >= 0 if s["ids"] is not None else torch.ones_like(w, dtype=torch.bool)
    h, w = torch.where(live[:, :, None], h, 0.0), torch.where(live, w, 0.0)
    out = [(h * w[:, :, None]).sum(1).to(s["h"].dtype)]
    if case["train"]:
        gy = s["gy"].float()
        out += [(w[:, :, None] * gy[:, None, :]).to(s["h"].dtype), torch.where(live, (h * gy[:, None, :]).sum(2), 0.0)]
    return out


def _plain(case, s):
    if case["op"] == "route":
        return _plain_route(case, s)
    if case["op"] == "dense":
        return [(_activation(s["x"], case["swiglu"]) @ _values(s["w"], s["ws"]).t()).to(s["x"].dtype)]
    return _plain_experts(case, s) if case["op"] == "experts" else _plain_combine(case, s)


# ------------------------------------------------------------------------------------------------- the framework's calls


def _framework(case, s):
    import quantized_matmul_amd as qm

    if case["op"] == "route":
        how = dict(score=case["score"], renormalize=case["renorm"], scale=case["scale"])
        weights, ids = qm.moe_route(s["logits"], case["k"], bias=s["bias"], groups=case["groups"],
                                    groups_kept=case["kept"], group_top=case["top"], **how)
        out = [weights, ids]
        if case["train"]:
            out.append(qm.moe_route_grad(s["logits"], ids, s["grad"], **how))
        return out
    if case["op"] == "combine":
        out = [qm.moe_combine(s["h"], s["weights"], s["ids"])]
        if case["train"]:
            out += qm.moe_combine_grad(s["gy"], s["h"], s["weights"], s["ids"])
        return out
    qw = qm.QuantizedWeight(s["w"], s["ws"], None, GROUP, 4, True, "mxfp4")
    activation = "swiglu" if case["swiglu"] else None
    if case["op"] == "dense":
        return [qm.mxfp4_matmul(s["x"], qw, activation=activation)]
    return [qm.gather_mxfp4_matmul(s["x"], qw, s["ids"], activation=activation)]


def run(state):
    return (_framework if own else _plain)(state["case"], state)


def work(case):
    op, size = case["op"], SIZE[case.get("dtype", "bf16")]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        rows = 3 if case["train"] else 1  # logits read for the choice and for the gradient, the gradient written
        return {"bytes": rows * T * E * size + T * k * (20 if case["train"] else 8) + (4 * E if case["bias"] else 0),
                "flops": T * E * (8 if case["train"] else 4)}
    if op == "combine":
        T, k, D = case["T"], case["k"], case["D"]
        if not case["train"]:
            return {"bytes": T * D * size * (k + 1) + T * k * 4, "flops": 2 * T * k * D}
        return {"bytes": T * D * size * (3 * k + 2) + T * k * 12, "flops": 5 * T * k * D}
    wide = 2 if case["swiglu"] else 1
    N, K = case["N"], case["K"]
    if op == "dense":
        M, hit = case["M"], 1
        read = M * K * wide * size
    else:
        M = case["T"] * case["k"]
        hit = min(case["E"], M)
        read = case["T"] * K * wide * size + M * 4
    return {"bytes": read + hit * N * (K // 2 + K // GROUP) + M * N * size, "flops": 2 * M * N * K}


# --------------------------------------------------------------------------------------------------------- 64-bit values


def _exact_values(words, scales):
    out = []
    for place in range(8):
        code = (words.long() >> (4 * place)) & 15
        power, half = (code >> 1) & 3, (code & 1).double()
        size = torch.where(power > 0, (1 + half / 2) * 2.0 ** (power - 1).double(), half / 2)
        out.append(torch.where(code >= 8, -size, size))
    v = torch.stack(out, -1)
    v = v.reshape(scales.shape + (GROUP,)) * (2.0 ** (scales.double() - 127))[..., None]
    return v.reshape(words.shape[:-1] + (-1,))


def _exact_rounded(x):
    """x in 64 bits rounded to mxfp4 along its last axis."""
    v = x.reshape(x.shape[:-1] + (-1, GROUP))
    most = v.abs().amax(-1, keepdim=True)
    unit = 2.0 ** ((torch.frexp(most)[1] - 3).clamp(-127, 127)).double()
    a = (v / unit).abs().clamp_max(6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    r = torch.sign(v) * torch.round(a / step) * step * unit  # round() takes a tie to even, which is the even code here
    return torch.where(most > 0, r, 0.0).reshape(x.shape)


def _exact_activation(case, x):
    x = x.double()
    if case["swiglu"]:
        half = x.shape[-1] // 2
        x = x[..., :half] * torch.sigmoid(x[..., :half]) * x[..., half:]
    return _exact_rounded(x)


def _exact_route(case, s):
    x = s["logits"].double()
    T, E, G, k, c = case["T"], case["E"], case["groups"], case["k"], case["scale"]
    dead = ~torch.isfinite(x)
    p = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(x, 1))
    key = (p + s["bias"].double() if case["bias"] else p).masked_fill(dead, -math.inf)
    if case["kept"] < G:
        inner = torch.sort(key.reshape(T, G, -1), dim=2, descending=True)[0][..., : case["top"]].sum(-1)
        order = torch.sort(inner, dim=1, descending=True, stable=True)[1]
        for place in range(case["kept"], G):
            out = order[:, place : place + 1] == torch.arange(E, device=x.device)[None] // (E // G)
            key = key.masked_fill(out, -math.inf)
    ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :k]
    live = key.gather(1, ids) > -math.inf
    q = p.clone().requires_grad_(False).gather(1, ids) * live
    total = q.sum(1, keepdim=True) if case["renorm"] else torch.ones((T, 1), device=x.device, dtype=x.dtype)
    total = torch.where(total > 0, total, 1.0)
    w = c * q / total
    out = [w, torch.where(live, ids, -1).to(torch.int32)]
    if case["train"]:
        g = s["grad"].double() * live
        # chain rule with the full Jacobians: weights by chosen scores, chosen scores by logits
        dq = c * g / total
        if case["renorm"]:
            dq = dq - (c * g * q).sum(1, keepdim=True) / total**2
        dq = dq * live
        full = torch.zeros_like(p).scatter_add_(1, ids, dq)
        if case["score"] == "sigmoid":
            gx = full * p * torch.sigmoid(-x)
        else:
            gx = p * (full - (full * p).sum(1, keepdim=True))
            if case["renorm"]:  # the two sums cancel for every logit outside the choice
                gx = gx * torch.zeros_like(p).scatter_add_(1, ids, live.double())
        out.append(torch.where(dead, 0.0, gx))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "combine":
        h, w = s["h"].double(), s["weights"].double()
        if s["ids"] is not None:
            w = w * (s["ids"] >= 0)
        y = torch.stack([(h[:, j] * w[:, j, None]) for j in range(case["k"])]).sum(0)
        if not case["train"]:
            return [y]
        gy = s["gy"].double()
        dw = torch.stack([(h[:, j] * gy).sum(1) for j in range(case["k"])], 1)
        if s["ids"] is not None:
            dw = dw * (s["ids"] >= 0)
        return [y, torch.stack([gy * w[:, j, None] for j in range(case["k"])], 1), dw]
    x = _exact_activation(case, s["x"])
    if case["op"] == "dense":
        return [torch.matmul(_exact_values(s["w"], s["ws"]), x.t().contiguous()).t().contiguous()]
    ids = s["ids"].reshape(-1)
    y = torch.zeros((ids.numel(), case["N"]), dtype=torch.float64, device=x.device)
    for e in range(case["E"]):
        rows = torch.nonzero(ids == e)[:, 0]
        if rows.numel():
            w = _exact_values(s["w"][e], s["ws"][e]).t().contiguous()
            y[rows] = torch.matmul(x[torch.div(rows, case["k"], rounding_mode="floor")], w)
    return [y.view(case["T"], case["k"], case["N"])]
