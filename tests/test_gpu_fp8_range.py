"""GPU: block-scaled e4m3 products at the ends of the range in which finite
inputs give finite results: the product of the two blocks' scales is finite in
fp32."""
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


# Powers of two: a block's codes are 448 and 0, its scale m / 448 rounded; 2^72 / 448 is under 2^63.2, so the product of
# two such scales is under 2^127.
BIG = 2.0 ** 72


@pytest.mark.parametrize("rows", [3, 300])  # the kernel for few rows, and the tensor cores'
def test_large_blocks_that_do_not_meet(z, rows):
    """Each factor's large value stands opposite a zero of the other: exact zeros, no NaN."""
    x = torch.zeros(rows, 256, device="cuda")
    x[:, 0] = BIG
    w = torch.zeros(1, 64, 256, device="cuda")
    w[:, :, 1] = BIG
    fp8 = z.BlockFp8()
    y = fp8.linear(x, fp8.quantize_weight(w), out_dtype=torch.float32)
    assert torch.equal(y, torch.zeros_like(y))
    # the gradients: dy's blocks against the weight's columns, and columns of dy and x with values in different rows
    grad = torch.zeros(rows, 64, device="cuda")
    grad[0, ::2] = BIG
    x = torch.zeros(rows, 256, device="cuda")
    x[1, :] = BIG
    w = torch.zeros(1, 64, 256, device="cuda")
    w[:, 1::2, :] = BIG
    dx, dw = fp8.linear_backward(grad, x, fp8.quantize_weight(w, backward=True), out_dtype=torch.float32)
    assert torch.equal(dx, torch.zeros_like(dx)) and torch.equal(dw, torch.zeros_like(dw))
    assert fp8.read_status() == z.OK


@pytest.mark.parametrize("rows", [3, 300])
def test_small_blocks(z, rows):
    """Scales whose product is just above the smallest normal number: (2^-54 / 448)^2 is above 2^-125.7."""
    tiny = 2.0 ** -54
    x = torch.full((rows, 128), tiny, device="cuda")
    w = torch.full((1, 64, 128), tiny, device="cuda")
    fp8 = z.BlockFp8()
    want = 128 * tiny * tiny
    y = fp8.linear(x, fp8.quantize_weight(w), out_dtype=torch.float32).double()
    # each scale m / 448 is rounded once, their product and its product with the codes' sum once each
    assert ((y / want - 1).abs() <= 5 * 2.0 ** -24).all()
    dx, dw = fp8.linear_backward(torch.full((rows, 64), tiny, device="cuda"), x,
                                 fp8.quantize_weight(w, backward=True), out_dtype=torch.float32)
    assert ((dx.double() / (64 * tiny * tiny) - 1).abs() <= 5 * 2.0 ** -24).all()
    # up to three blocks of rows, each added with a rounding of its own
    assert ((dw.double() / (rows * tiny * tiny) - 1).abs() <= 8 * 2.0 ** -24).all()
    assert fp8.read_status() == z.OK
