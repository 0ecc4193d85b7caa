"""GPU: the block-scaled e4m3 layer with few rows a group, at sizes where a CTA
works through many outputs, on both sides of the choice of its kernel.

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
    (1, 4000, 9000, 1, 0), (16, 1000, 20000, 1, 0), (33, 129, 257, 1, 0), (64, 1800, 5000, 1, 3), (65, 640, 700, 1, 0),
    (264, 2048, 1024, 64, 0), (40, 1800, 1100, 40, 7), (500, 700, 900, 33, 1), (1300, 640, 1000, 40, 40), (5, 8000, 128, 2, 0),
    (300, 128, 384, 100, 0), (20, 384, 130, 512, 2), (2600, 256, 516, 60, 0),
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
    packed = fp8.weight(w.to(torch.float8_e4m3fn), torch.ones(groups, -(-n // 128), -(-k // 128), device="cuda"))
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
    assert torch.equal(fp8.linear(x, packed, given), want.bfloat16())
