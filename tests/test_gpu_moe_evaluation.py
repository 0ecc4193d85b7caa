"""GPU: an evaluation of the example's block drops nothing, and its gradients are of what it computed."""
import pytest
import torch

from test_gpu_moe_layer import example, z  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 100])
def test_evaluation_of_a_block_with_dropout(example, tokens):  # noqa: F811
    args = dict(capacity=20, scale=0.7, seed=3)
    drops, plain = (example.MoeBlock(8, 2, 256, 128, dropout=p, **args) for p in (0.5, 0.0))
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x, grad_r, grad_h = (torch.randn(tokens, 256, generator=g, device="cuda").bfloat16() for _ in range(3))
    want = (*plain.forward(x), *plain.backward(grad_r, grad_h))
    trained = drops.forward(x, step=1)
    got = (*drops.forward(x, step=1, train=False), *drops.backward(grad_r, grad_h))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not torch.equal(trained[0], got[0])
    drops.check_status()
