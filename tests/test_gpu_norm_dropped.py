"""GPU: what is dropped has no part in the gradients, whatever its own gradient is, in each of
the kernels that hold a row."""
import pytest
import torch

import norm_ref as ref
from gpu_util import load_lib, require_gpu

pytestmark = pytest.mark.gpu
B, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def z():
    require_gpu()
    load_lib()
    import lossless_bf16_exponent_split_gb300 as z
    return z


# a row held by part of a warp, a warp, a CTA, clusters of two and four, and read several times; on and off 16 bytes
@pytest.mark.parametrize("hidden", [64, 255, 256, 2048, 2047, 9600, 16384, 16383, 16385, 16392])
@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_gradients_that_overflowed_where_the_mask_drops(z, hidden, dtype, bad):
    rows, g = 6, torch.Generator(device="cuda").manual_seed(hidden)
    x, y, grad_r, grad_h = (torch.randn(rows, hidden, generator=g, device="cuda").to(dtype) for _ in range(4))
    w, gate = torch.rand(hidden, generator=g, device="cuda"), torch.rand(2, hidden, generator=g, device="cuda").to(dtype)
    n = z.ResidualNorm(hidden, dropout=0.5, seed=4)
    keep = ref.kept(rows, hidden, 0.5, 4, 0).cuda()
    r, _ = n.add(x, y, w, gate=gate)
    spoilt = torch.where(keep, grad_r, torch.full_like(grad_r, bad))
    for gh, weight in ((grad_h, w), (None, None)):
        want = n.add_backward(grad_r, gh, r, y, weight, gate=gate)
        got = n.add_backward(spoilt, gh, r, y, weight, gate=gate)
        assert torch.equal(got.y, want.y) and bool((got.y[~keep] == 0).all())
        assert torch.equal(got.gate, want.gate) and (gh is None or torch.equal(got.weight, want.weight))
        assert torch.equal(got.x[keep], want.x[keep]) and not bool(got.x[~keep].isfinite().any())


@pytest.mark.parametrize("hidden", [64, 255, 2048, 2047, 9600, 16383, 16385, 16392])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_values_that_the_mask_drops_may_be_anything(z, hidden, bad):
    rows, g = 6, torch.Generator(device="cuda").manual_seed(hidden)
    x, y, grad_r, grad_h = (torch.randn(rows, hidden, generator=g, device="cuda").to(B) for _ in range(4))
    w, gate = torch.rand(hidden, generator=g, device="cuda"), torch.rand(2, hidden, generator=g, device="cuda")
    n = z.ResidualNorm(hidden, dropout=0.5, seed=4)
    keep = ref.kept(rows, hidden, 0.5, 4, 0).cuda()
    spoilt = torch.where(keep, y, torch.full_like(y, bad))
    r, h = n.add(x, y, w, gate=gate)
    assert all(torch.equal(a, b) for a, b in zip(n.add(x, spoilt, w, gate=gate), (r, h)))
    for a, b in zip(n.add_backward(grad_r, grad_h, r, spoilt, w, gate=gate), n.add_backward(grad_r, grad_h, r, y, w, gate=gate)):
        assert (a is None and b is None) or torch.equal(a, b)
