"""GPU: the block-scaled e4m3 layer where most tiles of a product have nothing to
sum: many groups without rows, and long tails of rows outside every group.  A CTA
then goes through one tile after another without a block of the reduction, and
the tile before them must still end."""
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


@pytest.mark.parametrize("sizes,tail,k,n", [
    ([2] + [0] * 36, 0, 340, 3936), ([0] * 20 + [30, 20] + [0] * 16, 0, 1500, 1248), ([1] * 60, 0, 520, 2000), ([200, 100], 40000, 256, 1030),
    ([130], 30001, 128, 2048), ([0, 0, 0], 20000, 200, 1000), ([129, 0, 0, 0, 0, 0, 500] + [0] * 60, 5000, 800, 900),
])
def test_values_and_no_waits_run_out(z, sizes, tail, k, n):
    rows, groups = sum(sizes) + tail, len(sizes)
    gen = torch.Generator(device="cuda").manual_seed(rows + k)
    ends = torch.tensor([0] + sizes).cumsum(0)
    offsets = ends.int().cuda()

    # whole numbers below 9 and a largest value of 448 in each block of a row and of a column: scales are one, sums exact
    def whole(cols):
        v = torch.randint(-3, 4, (rows, cols), generator=gen, device="cuda").float()
        v[:, ::128] = 448.0
        for lo in ends[:-1].tolist():
            if lo < rows:
                v[lo] = 448.0
        for lo, hi in zip(ends[:-1].tolist(), ends[1:].tolist()):
            v[lo:hi:128] = 448.0
        return v.bfloat16()

    x, grad = whole(k), whole(n)
    w = torch.randint(-2, 3, (groups, n, k), generator=gen, device="cuda").float()
    fp8 = z.BlockFp8()
    packed = fp8.weight(w.to(torch.float8_e4m3fn), torch.ones(groups, -(-n // 128), -(-k // 128), device="cuda"), backward=True)
    y = fp8.linear(x, packed, offsets, out_dtype=torch.float32)
    dx, dw = fp8.linear_backward(grad, x, packed, offsets, out_dtype=torch.float32)
    assert fp8.read_status() == z.OK
    live = int(ends[-1])
    assert not y[live:].any() and not dx[live:].any()
    for g, (lo, hi) in enumerate(zip(ends[:-1].tolist(), ends[1:].tolist())):
        a, b = x[lo:hi].double(), grad[lo:hi].double()
        assert torch.equal(y[lo:hi].double(), a @ w[g].double().t())
        assert torch.equal(dx[lo:hi].double(), b @ w[g].double())
        # squares of 448 leave the 24 bits: the bound is the sum's rounding
        want = b.t() @ a
        assert ((dw[g].double() - want).abs() <= 2.0 ** -20 * (b.abs().t() @ a.abs())).all()
