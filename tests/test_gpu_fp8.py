"""GPU: the block-scaled e4m3 layers against 64-bit numpy on the same quantised
values, at odd sizes, ragged and empty groups, strides and special values."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
from gpu_util import load_lib, require_gpu

pytestmark = pytest.mark.gpu

# The instruction multiplies codes exactly and adds the 128 products of a block into an fp32 accumulator whose
# alignment keeps at least 2^-22 of its largest term; blocks are added in fp32 (2^-24 each), after two scale products.
# All of it is bounded by the sum of the terms' magnitudes.
def bound(size, blocks):
    return size * (2.0 ** -18 + (blocks + 4) * 2.0 ** -23)


@pytest.fixture(scope="module")
def z():
    require_gpu()
    load_lib()
    import lossless_bf16_exponent_split_gb300 as z
    return z


def offsets_of(rng, rows, groups, tail):
    cuts = np.sort(rng.integers(0, rows - tail + 1, groups - 1)) if groups > 1 else np.zeros(0, np.int64)
    return np.concatenate([[0], cuts, [rows - tail]]).astype(np.int32)


def data(rng, shape, dtype):
    x = rng.normal(size=shape) * np.exp(rng.normal(size=(shape[0],) + (1,) * (len(shape) - 1)))
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


CASES = [  # rows, k, n, groups, tail, type
    (1, 4096, 512, 1, 0, torch.bfloat16), (1, 1, 1, 1, 0, torch.float32), (7, 129, 17, 1, 0, torch.float32),
    (33, 1000, 130, 3, 2, torch.bfloat16), (70, 300, 65, 40, 5, torch.float32), (31, 257, 31, 2, 0, torch.bfloat16),
    (128, 128, 256, 1, 0, torch.bfloat16), (129, 256, 256, 1, 0, torch.bfloat16), (200, 200, 1000, 1, 0, torch.float32),
    (700, 515, 333, 5, 19, torch.bfloat16), (1500, 2048, 384, 4, 0, torch.bfloat16), (2111, 77, 259, 12, 300, torch.bfloat16),
    (4096, 640, 64, 64, 1, torch.bfloat16), (1300, 136, 2064, 1, 0, torch.float32),
]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,k,n,groups,tail,dtype", CASES)
def test_linear_and_gradients(z, rows, k, n, groups, tail, dtype, out):
    rng = np.random.default_rng(rows + k + n)
    off = offsets_of(rng, rows, groups, tail)
    x, grad = data(rng, (rows, k), dtype), data(rng, (rows, n), dtype)
    w = torch.from_numpy((rng.normal(size=(groups, n, k)) * k ** -0.5).astype(np.float32))
    fp8 = z.BlockFp8()
    packed = fp8.quantize_weight(w.cuda(), backward=True)
    q, s, full = ref.weight(w.numpy())
    offd = None if groups == 1 and tail == 0 else torch.from_numpy(off).cuda()
    slack = 2.0 ** -8 if out == torch.bfloat16 else 2.0 ** -23

    def close(got, want, size, blocks):
        got = got.double().cpu().numpy()
        assert (np.abs(got - want) <= bound(size, blocks) + slack * np.abs(want)).all()

    y = fp8.linear(x.cuda(), packed, offd, out_dtype=out)
    want, size = ref.linear(x.float().numpy(), full, off)
    close(y, want, size, -(-k // 128))
    assert not y[rows - tail:].any()

    dx, dw = fp8.linear_backward(grad.cuda(), x.cuda(), packed, offd, out_dtype=out)
    want, size = ref.linear(grad.float().numpy(), full.transpose(0, 2, 1), off)
    close(dx, want, size, -(-n // 128))
    assert not dx[rows - tail:].any()
    want, size = ref.weight_grad(grad.float().numpy(), x.float().numpy(), off)
    close(dw, want, size, -(-rows // 128))
    assert fp8.read_status() == z.OK

    # the same weight given as codes and scales
    same = fp8.weight(torch.from_numpy(q).to(torch.float8_e4m3fn).cuda(), torch.from_numpy(s.astype(np.float32)).cuda(), backward=True)
    assert torch.equal(same.packed, packed.packed) and torch.equal(same.packed_t, packed.packed_t)


def test_gradients_against_differences(z):
    """On values that e4m3 holds exactly under every scale in play (powers of two), the layer is linear and its gradients
    are those of sum(grad * linear(x, w)) by differences."""
    rng = np.random.default_rng(1)
    rows, k, n = 140, 96, 80

    def powers(*shape):
        p = np.exp2(rng.integers(-2, 3, shape)) * rng.choice([-1.0, 1.0], shape)
        p.reshape(-1)[:: 7] = 448.0 / 112  # 4: every block's largest value, so every scale is a power of two times 4 / 448
        return p.astype(np.float32)

    x, w, grad = powers(rows, k), powers(1, n, k), powers(rows, n)
    fp8 = z.BlockFp8()

    def loss(x, w):
        y = fp8.linear(torch.from_numpy(x).cuda(), fp8.quantize_weight(torch.from_numpy(w).cuda()), out_dtype=torch.float32)
        return float((y.double().cpu().numpy() * grad).sum())

    dx, dw = fp8.linear_backward(torch.from_numpy(grad).cuda(), torch.from_numpy(x).cuda(),
                                 fp8.quantize_weight(torch.from_numpy(w).cuda(), backward=True), out_dtype=torch.float32)
    dx, dw = dx.double().cpu().numpy(), dw.double().cpu().numpy()
    # the layer's error in 32 bits, summed over the outputs that a changed value reaches, over the difference's width
    scale = np.abs(x).max() * np.abs(w).max() * np.abs(grad).max() * k * (2.0 ** -18 + 5 * 2.0 ** -23)
    for at in [(0, 0), (13, 95), (139, 50)]:
        hi, lo = x.copy(), x.copy()
        hi[at], lo[at] = 2.0, -2.0
        assert abs((loss(hi, w) - loss(lo, w)) / 4.0 - dx[at]) <= 2 * n * scale
    for at in [(0, 0, 0), (0, 79, 3), (0, 41, 95)]:
        hi, lo = w.copy(), w.copy()
        hi[at], lo[at] = 2.0, -2.0
        assert abs((loss(x, hi) - loss(x, lo)) / 4.0 - dw[at]) <= 2 * rows * scale


@pytest.mark.parametrize("rows", [3, 300])
def test_exact_on_small_whole_numbers(z, rows):
    """Codes of whole numbers under scale one: every product and sum is exact in fp32, so is the layer."""
    rng = np.random.default_rng(2)
    k, n = 512, 300
    x = rng.integers(-8, 9, (rows, k)).astype(np.float32)
    w = rng.integers(-8, 9, (1, n, k)).astype(np.float32)
    x[:, ::128] = 448.0
    fp8 = z.BlockFp8()
    packed = fp8.weight(torch.from_numpy(w).to(torch.float8_e4m3fn).cuda(), torch.ones(1, 3, 4, device="cuda"), backward=True)
    y = fp8.linear(torch.from_numpy(x).cuda(), packed, out_dtype=torch.float32)
    assert np.array_equal(y.double().cpu().numpy(), x.astype(np.float64) @ w[0].T.astype(np.float64))


@pytest.mark.parametrize("rows", [9, 260])
def test_special_values_stay_in_their_rows(z, rows):
    k, n = 300, 140
    rng = np.random.default_rng(4)
    x = data(rng, (rows, k), torch.bfloat16)
    x[2] = 0.0
    x[3, 5] = float("nan")
    x[4, 299] = float("inf")
    x[5] = 2.0 ** -120  # below the smallest largest magnitude: codes of zero
    x[6, 7] = 1.0e37
    w = torch.from_numpy((rng.normal(size=(1, n, k))).astype(np.float32))
    fp8 = z.BlockFp8()
    packed = fp8.quantize_weight(w.cuda(), backward=True)
    y = fp8.linear(x.cuda(), packed, out_dtype=torch.float32).cpu()
    assert y[3].isnan().all() and y[4].isnan().all()
    assert not y[2].any() and not y[5].any()
    keep = [r for r in range(rows) if r not in (3, 4)]
    assert torch.isfinite(y[keep]).all()
    want, size = ref.linear(x[keep].float().numpy(), ref.weight(w.numpy())[2], [0, len(keep)])
    assert (np.abs(y[keep].double().numpy() - want) <= bound(size, 3) + 2.0 ** -23 * np.abs(want)).all()
    dw = fp8.linear_backward(data(rng, (rows, n), torch.bfloat16).cuda(), x.cuda(), packed, input_grad=False)[1][0].cpu()
    bad = dw.isnan().all(0)
    assert bad[5] and bad[299] and bad.sum() == 2 and dw[:, ~bad].isfinite().all()


@pytest.mark.parametrize("rows,groups", [(60, 4), (900, 4)])
def test_strided_rows(z, rows, groups):
    rng = np.random.default_rng(6)
    wide, up = data(rng, (rows, 777), torch.bfloat16).cuda(), data(rng, (rows, 500), torch.bfloat16).cuda()
    fp8 = z.BlockFp8()
    packed = fp8.quantize_weight(torch.randn(groups, 200, 264, device="cuda"), backward=True)
    off = torch.from_numpy(offsets_of(rng, rows, groups, 0)).cuda()
    for lo in (0, 3, 8):  # odd and aligned first columns
        x, g = wide[:, lo:lo + 264], up[:, lo:lo + 200]
        assert torch.equal(fp8.linear(x, packed, off), fp8.linear(x.contiguous(), packed, off))
        for a, b in zip(fp8.linear_backward(g, x, packed, off), fp8.linear_backward(g.contiguous(), x.contiguous(), packed, off)):
            assert torch.equal(a, b)


def test_no_rows_and_empty_groups(z):
    fp8 = z.BlockFp8()
    packed = fp8.quantize_weight(torch.randn(3, 40, 56, device="cuda"), backward=True)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, g = torch.empty(0, 56, device="cuda"), torch.empty(0, 40, device="cuda")
    assert fp8.linear(x, packed, off).shape == (0, 40)
    dx, dw = fp8.linear_backward(g, x, packed, off)
    assert dx.shape == (0, 56) and not dw.any()
    for rows in (20, 500):  # rows, but none in any group
        x, g = torch.randn(rows, 56, device="cuda"), torch.randn(rows, 40, device="cuda")
        assert not fp8.linear(x, packed, off).any()
        dx, dw = fp8.linear_backward(g, x, packed, off)
        assert not dx.any() and not dw.any()


@pytest.mark.parametrize("table", [[0, -5, 900, 40], [0, 400, 10, 400], [0, 2147483647, -2147483648, 7], [500, 400, 300, 200]])
@pytest.mark.parametrize("rows", [50, 400])
def test_bad_offsets_stay_in_bounds(z, table, rows):
    """A table that is no table of groups gives some output, and touches nothing outside its tensors."""
    fp8 = z.BlockFp8()
    packed = fp8.quantize_weight(torch.randn(3, 40, 56, device="cuda"), backward=True)
    off = torch.tensor(table, dtype=torch.int32, device="cuda")
    x, g = torch.randn(rows, 56, device="cuda"), torch.randn(rows, 40, device="cuda")
    fp8.linear(x, packed, off)
    fp8.linear_backward(g, x, packed, off)
    torch.cuda.synchronize()
    assert fp8.read_status() == z.OK


def test_refusals(z):
    fp8 = z.BlockFp8()
    w = fp8.quantize_weight(torch.randn(2, 40, 56, device="cuda"))
    x, off = torch.randn(5, 56, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    for call in (lambda: fp8.linear(x, w), lambda: fp8.linear(x[:, :55], w, off), lambda: fp8.linear(x.double(), w, off),
                 lambda: fp8.linear(x.T, w, off), lambda: fp8.linear(x, w, off[:2]), lambda: fp8.linear(x, w, off.long()),
                 lambda: fp8.linear(x, w, off, out_dtype=torch.float16), lambda: fp8.linear_backward(x[:, :40], x, w, off),
                 lambda: fp8.linear_backward(x[:4, :40], x, w, off, input_grad=False),
                 lambda: fp8.linear_backward(x[:, :40].bfloat16(), x, w, off, input_grad=False),
                 lambda: fp8.weight(torch.zeros(1, 4, 4, device="cuda"), torch.ones(1, 1, 1, device="cuda")),
                 lambda: fp8.weight(torch.zeros(1, 4, 4, device="cuda").to(torch.float8_e4m3fn), torch.ones(1, 2, 1, device="cuda"))):
        with pytest.raises(ValueError):
            call()
