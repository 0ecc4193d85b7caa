"""GPU: the weight gradient of the block-scaled e4m3 layer where the sum over a
group's rows is cut into parts that several CTAs take.

Columns of whole numbers with a largest value of 448 in every block of 128 rows:
scales are one, and every sum is below 2^24 and exact in fp32."""
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


@pytest.mark.parametrize("cuts,k,n,tail", [
    ([3200], 64, 64, 0), ([5000], 300, 260, 0), ([0, 6400, 6400, 9999], 100, 40, 31), ([4000, 4100], 520, 129, 0),
    ([1, 2, 9000], 256, 128, 0), ([3583], 1000, 700, 2),
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_exact(z, cuts, k, n, tail, dtype):
    rows, groups = cuts[-1] + tail, len(cuts)
    gen = torch.Generator(device="cuda").manual_seed(rows + k)

    def whole(cols):
        v = torch.randint(-4, 5, (rows, cols), generator=gen, device="cuda").float()
        lo = 0
        for hi in cuts:
            v[lo:hi:128] = 448.0
            lo = hi
        return v.to(dtype)

    x, grad = whole(k), whole(n)
    fp8 = z.BlockFp8()
    weight = fp8.quantize_weight(torch.zeros(groups, n, k, device="cuda"), backward=True)
    offsets = torch.tensor([0, *cuts], dtype=torch.int32, device="cuda")
    given = None if groups == 1 and tail == 0 else offsets
    for input_grad in (False, True):
        dx, dw = fp8.linear_backward(grad, x, weight, given, input_grad=input_grad, out_dtype=torch.float32)
        lo = 0
        for g, hi in enumerate(cuts):
            assert torch.equal(dw[g].double(), grad[lo:hi].double().t() @ x[lo:hi].double()), (input_grad, g)
            lo = hi
        assert dx is None or not dx.any()
    assert fp8.read_status() == z.OK
