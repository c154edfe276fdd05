"""Routing of many tokens with groups that are not whole lanes, against the
64-bit statement (moe_reference).

A wave keeps the row of such a group choice in its own LDS, next to the other
waves' places: only launches of several workgroups, with waves out of step, and
tokens of every wave of a workgroup can show one wave in another's.

Tokens are kept whose choice is clear in 64 bits: of the keys and of the
groups' keys that fp32 sums, no two are nearer than 5e-6. A sigmoid is within
4 * 2^-24 of its 64-bit value and a token's softmax scores, of up to 500
experts, together within 14 * 2^-24; a key below 2 adds a rounding of 2^-24, a
sum of two one of 2^-23: a group's key is within 1.2e-6, and a comparison has
two. Weights: 4e-6 relative, as for every route.
"""
import numpy as np
import pytest
import torch

import moe_reference as ref

pytestmark = pytest.mark.gpu

qm = pytest.importorskip("quantized_matmul_amd")

DEV = "cuda:0"


def clear_tokens(x, k, score, bias, groups, kept, top):
    """Rows of x whose choice hangs on no rounding, repeated to x's length."""
    s = ref.scores(x, score)
    key = s if bias is None else s + bias
    key = np.where(np.isfinite(x), key, -1e6 * (1 + np.arange(x.shape[1])))   # masked ones: never near
    near = np.zeros(len(x), bool)
    if top == 2 or bias is not None:
        g = np.sort(key.reshape(len(x), groups, -1), axis=2)[:, :, -top:].sum(2)
        near |= (np.diff(np.sort(g, axis=1), axis=1) < 5e-6).any(1)
    if bias is not None:
        near |= (np.diff(np.sort(key, axis=1), axis=1) < 5e-6).any(1)
    clear = np.flatnonzero(~near)
    assert len(clear) >= 500
    return x[np.resize(clear, len(x))]


@pytest.mark.parametrize("E,groups,kept,k", [(24, 8, 3, 6), (36, 4, 2, 8), (40, 8, 5, 4), (48, 4, 1, 8), (60, 4, 2, 8),
                                             (60, 6, 3, 16), (60, 20, 7, 8), (63, 7, 3, 5), (100, 10, 4, 8),
                                             (300, 12, 5, 9)])
@pytest.mark.parametrize("score,bias,top", [("softmax", False, 1), ("sigmoid", False, 2), ("sigmoid", True, 2),
                                            ("softmax", True, 1)])
def test_route_many_tokens_in_odd_groups(E, groups, kept, k, score, bias, top):
    T = 6001
    print(f"route T{T} E{E} k{k} {score} groups {groups}/{kept}/{top} bias {bias}", flush=True)
    rng = np.random.default_rng(1000 * E + groups)
    b = rng.normal(size=E).astype(np.float32) * np.float32(0.05) if bias else None
    x = rng.normal(size=(T, E)).astype(np.float32) * np.float32(1.5)
    x[::2] -= np.float32(8.0) if not (bias or top == 2) else np.float32(0.5)    # rows of negative logits
    x = clear_tokens(x.astype(np.float64), k, score, b, groups, kept, top)
    t = torch.from_numpy(x).float().to(DEV)
    w, ids = qm.moe_route(t, k, score=score, bias=None if b is None else torch.from_numpy(b).to(DEV), groups=groups,
                          groups_kept=kept, group_top=top)
    rw, rids = ref.route(x, k, score, bias=b, groups=groups, groups_kept=kept, group_top=top)
    np.testing.assert_array_equal(ids.cpu().numpy(), rids)
    np.testing.assert_allclose(w.cpu().double().numpy(), rw, rtol=4e-6)


@pytest.mark.parametrize("E,groups,kept,top,k", [(64, 1, 1, 1, 8), (60, 4, 2, 2, 8), (64, 4, 2, 2, 8), (256, 8, 4, 2, 8),
                                                 (48, 16, 5, 1, 6), (500, 10, 3, 2, 40)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masked_experts_with_bias_and_groups(E, groups, kept, top, k, score):
    """Masks at random, whole groups masked, groups with fewer experts than their key counts, rows without any."""
    T = 2003
    print(f"route T{T} E{E} k{k} {score} groups {groups}/{kept}/{top} masked", flush=True)
    rng = np.random.default_rng(2000 * E + groups)
    b = rng.normal(size=E).astype(np.float32) * np.float32(0.5)
    x = (rng.normal(size=(T, E)).astype(np.float32) * np.float32(1.5)).astype(np.float64)
    x = clear_tokens(x, k, score, b, groups, kept, top)
    per = E // groups
    x[rng.random((T, E)) < rng.choice([0.0, 0.3, 0.95], (T, 1))] = -np.inf
    x[rng.random((T, groups)).repeat(per, 1) < rng.choice([0.0, 0.5], (T, 1))] = np.nan
    x[::50] = -np.inf
    x[1::50, per:] = -np.inf
    x = clear_tokens(x, k, score, b, groups, kept, top)
    t, how = torch.from_numpy(x).float().to(DEV), dict(groups=groups, groups_kept=kept, group_top=top)
    w, ids = qm.moe_route(t, k, score=score, bias=torch.from_numpy(b).to(DEV), **how)
    rw, rids = ref.route(x, k, score, bias=b, **how)
    assert (rids[:, 0] < 0).any() and (rids[:, -1] >= 0).any()
    np.testing.assert_array_equal(ids.cpu().numpy(), rids)
    np.testing.assert_allclose(w.cpu().double().numpy(), rw, rtol=4e-6)
