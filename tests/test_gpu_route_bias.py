"""GPU: a NaN bias refuses the rows whose expert it belongs to is available in,
and no others."""
import pytest
import torch

from gpu_util import load_lib, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def z():
    require_gpu()
    load_lib()
    import lossless_bf16_exponent_split_gb300 as z
    return z


@pytest.mark.parametrize("tokens", [3, 4500])  # a warp a token, and several tokens a warp
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_bias(z, tokens, score):
    inf, nan = float("inf"), float("nan")
    moe = z.Moe(4, 2, score=score)
    bias = torch.tensor([0.0, nan, 0.0, 0.0], device="cuda")
    l = torch.tensor([1.0, -inf, 2.0, 3.0], device="cuda").repeat(tokens, 1)
    idx, _ = moe.route(l, bias)
    assert torch.equal(idx, torch.tensor([[3, 2]], dtype=torch.int32, device="cuda").expand(tokens, 2))
    assert moe.read_status() == z.OK
    l[1, 1] = 0.0
    idx, w = moe.route(l, bias)
    assert idx[1].tolist() == [-1, -1] and w[1].tolist() == [0.0, 0.0]
    assert idx[0].tolist() == [3, 2] and idx[2:].tolist() == [[3, 2]] * (tokens - 2)
    assert moe.read_status() == z.INVALID_ARG
