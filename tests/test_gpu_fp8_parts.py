"""GPU: the block-scaled e4m3 layer and its input's gradient where a tile's
reduction is cut into parts that several CTAs sum and one joins.

x's blocks have a largest value of 448 and the weights' scales are one, so codes
are the whole numbers themselves, every product and sum is one below 2^24, and
the result is exact in fp32 whatever the order of its sums."""
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


@pytest.mark.parametrize("rows,k,n,groups,tail", [
    (100, 4096, 1000, 1, 0), (128, 1800, 512, 1, 0), (200, 2048, 300, 3, 5), (48, 14336, 520, 1, 0), (257, 1025, 129, 1, 0),
    (130, 1100, 2000, 5, 0), (33, 4096, 4096, 1, 1), (600, 1536, 256, 4, 0), (900, 8000, 250, 2, 100),
])
def test_exact(z, rows, k, n, groups, tail):
    gen = torch.Generator(device="cuda").manual_seed(rows + k)

    def whole(*shape):
        return torch.randint(-8, 9, shape, generator=gen, device="cuda").float()

    x, w = whole(rows, k), whole(groups, n, k)
    x[:, ::128] = 448.0
    cuts = torch.randint(0, rows - tail + 1, (groups - 1,), generator=gen, device="cuda").sort().values
    ends = torch.tensor([0, rows - tail], device="cuda")
    offsets = torch.cat([ends[:1], cuts, ends[1:]]).int()
    fp8 = z.BlockFp8()
    packed = fp8.weight(w.to(torch.float8_e4m3fn), torch.ones(groups, -(-n // 128), -(-k // 128), device="cuda"), backward=True)
    given = None if groups == 1 and tail == 0 else offsets
    y = fp8.linear(x, packed, given, out_dtype=torch.float32)
    assert fp8.read_status() == z.OK
    bounds = offsets.tolist()
    want = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    for g in range(groups):
        lo, hi = bounds[g], bounds[g + 1]
        if hi > lo:
            want[lo:hi] = x[lo:hi].double() @ w[g].double().t()
    assert torch.equal(y.double(), want)
    # twice: the counters of the first call are ready for the second
    assert torch.equal(fp8.linear(x, packed, given).double(), want.bfloat16().double())
    # the gradient of another layer's input, whose output x is
    turned = fp8.weight(w.transpose(1, 2).contiguous().to(torch.float8_e4m3fn),
                        torch.ones(groups, -(-k // 128), -(-n // 128), device="cuda"), backward=True)
    other = torch.zeros(rows, n, device="cuda")
    dx, _ = fp8.linear_backward(x, other, turned, given, weight_grad=False, out_dtype=torch.float32)
    assert torch.equal(dx.double(), want)
    both, dw = fp8.linear_backward(x.bfloat16(), other.bfloat16(), turned, given, out_dtype=torch.float32)
    assert torch.equal(both.double(), want) and not dw.any()
    assert fp8.read_status() == z.OK
