"""The example layer: its pass through the operators against their 64-bit
statements, and the training of its router.

The forward pass is compared with the statement fed the kernels' own
intermediate values, so that no expert changes hands: products and the
activation's 4-bit codes round as in test_gpu_moe, the combine once more."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import moe_reference as ref

pytestmark = pytest.mark.gpu

qm = pytest.importorskip("quantized_matmul_amd")


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer_example", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def f64(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("T", [1, 33])
def test_forward_and_gate_gradient(example, T):
    layer = example.random_layer(8, 3, 96, 64)
    x = torch.randn(T, 96, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    y, (_, logits, weights, ids, o) = layer.forward(x)
    rw, rids = ref.route(f64(logits), 3, "sigmoid", bias=f64(layer.bias))
    np.testing.assert_array_equal(ids.cpu().numpy(), rids)
    np.testing.assert_allclose(f64(weights), rw, rtol=4e-6)
    ry = ref.combine(f64(o), f64(weights), rids)
    assert (np.abs(f64(y) - ry) <= 2.0 ** -8 * np.abs(ry) + 1e-5).all()
    gy = torch.randn(T, 96, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    grad = layer.gate_gradient(layer.forward(x)[1], gy)
    _, rgw = ref.combine_grad(f64(gy), f64(o), f64(weights), rids)
    rg = ref.route_grad(f64(logits), rids, rgw, "sigmoid", True, 1.0).T @ f64(x)
    assert np.abs(f64(grad) - rg).max() <= 1e-4 * np.abs(rg).max()


def test_router_learns_and_loads_even_out(example):
    layer = example.random_layer(16, 4, 256, 128)
    teacher = layer.gate.clone()
    noise = torch.randn(teacher.shape, generator=torch.Generator().manual_seed(5)).cuda()
    layer.gate = teacher + 0.5 * teacher.std() * noise
    losses = example.train_router(layer, teacher, 2048, 20)
    assert losses[-1] < 0.5 * losses[0], losses
    layer.gate[0] *= 3.0                                  # one expert with far larger scores, both ways
    layer.gate[0] += 0.2
    x = (torch.randn(2048, 256, generator=torch.Generator().manual_seed(6)) + 0.5).bfloat16().cuda()
    first = layer.balance(layer.forward(x)[1][3], 0.02)
    for _ in range(60):
        last = layer.balance(layer.forward(x)[1][3], 0.02)
    assert last < first and last < 1.5, (first, last)


def test_command(example, capsys):
    losses = example.main(["--tokens", "300", "--experts", "8", "--choice", "2", "--dim", "128", "--width", "64",
                           "--steps", "3"])
    assert len(losses) == 3 and all(np.isfinite(losses))
    assert "forward, 300 tokens" in capsys.readouterr().out
