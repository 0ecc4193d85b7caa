"""GPU: dropout against the generator's plain form, bit for bit: a kept value is
one product, rounded once more to 16 bits."""
import numpy as np
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


def expected(x, p, seed, offset):
    k = ref.kept(*x.shape, p, seed, offset)
    f = x.cpu().float() * torch.tensor(ref.gain(p), dtype=torch.float32)
    return torch.where(k, f, 0.0).to(x.dtype)


@pytest.mark.parametrize("rows,cols,dtype,p,seed,offset", [
    (1, 1, B, 0.5, 0, 0), (1, 8, B, 0.1, 1, 1), (3, 7, F, 0.3, 2, 1 << 40), (33, 1024, B, 0.1, (1 << 64) - 1, (1 << 64) - 1),
    (100, 2047, F, 0.5, 77, 5), (257, 255, B, 0.25, 3, 9), (5000, 24, B, 0.1, 4, 1), (70000, 3, F, 0.2, 5, 2), (9, 20000, B, 0.9, 6, 3),
    (2, 131072, F, 0.05, 8, 4), (1000, 264, F, 0.00002, 9, 5), (64, 256, B, 0.0, 9, 5), (64, 256, F, 1.0, 9, 5), (3, 100, B, 0.999999, 1, 1),
    (700, 511, B, 0.1, 1 << 63, 7)])
def test_dropout(z, rows, cols, dtype, p, seed, offset):
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g, device="cuda").to(dtype)
    drop = z.Dropout(p, seed=seed)
    want = expected(x, p, seed, offset)
    out = drop.apply(x, offset)
    assert torch.equal(out.cpu(), want)
    assert torch.equal(drop.apply(x, torch.tensor([offset - (1 << 64) if offset >> 63 else offset], device="cuda")).cpu(), want)
    for pad in (8, 3):  # rows of a wider matrix, on and off 16 bytes
        wide = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")[:, :cols]
        wide.copy_(x)
        assert torch.equal(drop.apply(wide, offset).cpu(), want)
    assert torch.equal(drop.apply(x, offset, out=x).cpu(), want) and torch.equal(x.cpu(), want)


def test_what_is_dropped_may_hold_anything(z):
    keep = ref.kept(64, 512, 0.5, 3, 0)
    x = torch.where(keep, 1.0, float("nan")).cuda()
    assert torch.equal(z.Dropout(0.5, seed=3).apply(x).cpu(), torch.where(keep, 2.0, 0.0))


def test_nothing_is_written_outside(z):
    for rows, cols in ((3, 9), (5, 264), (7, 1001)):
        for dtype, code in ((B, z.BF16), (F, z.F32)):
            x = torch.randn(rows, cols, device="cuda").to(dtype)
            out = torch.full((rows * cols + 512,), 7.0, dtype=dtype, device="cuda")
            assert z.zccl_dropout(x.data_ptr(), code, cols, rows, cols, 0.3, 5, 6, None, out.data_ptr() + 256 * out.element_size(),
                                  torch.cuda.current_stream().cuda_stream) == z.OK
            assert bool((out[:256] == 7).all()) and bool((out[256 + rows * cols:] == 7).all())
            assert torch.equal(out[256:256 + rows * cols].view(rows, cols).cpu(), expected(x, 0.3, 5, 6))


def test_rows_beyond_2_to_31_values(z):
    """Addresses and rows of a matrix of more than 2^31 values."""
    rows, cols = (1 << 21) + 3, 1032
    x = torch.ones(rows, cols, dtype=B, device="cuda")
    out = z.Dropout(0.5, seed=1).apply(x, 2, out=x)
    block = np.arange(rows - 5, rows, dtype=np.uint64)
    words = ref.philox((np.full(5, 128, np.uint64), block, np.full(5, 2, np.uint64), np.zeros(5, np.uint64)), (1, 0))
    halves = np.stack([np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1) for w in words], -2).reshape(5, 8)
    assert torch.equal(out[-5:, 1024:].float().cpu(), torch.from_numpy(np.where(halves >= 32768, 2.0, 0.0)).float())


def test_masks_of_a_graph(z):
    drop = z.Dropout(0.5, seed=11)
    x = torch.ones(40, 136, dtype=B, device="cuda")
    offset = torch.zeros(1, dtype=torch.int64, device="cuda")
    drop.apply(x, offset)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = drop.apply(x, offset)
        offset += 1
    for i in range(3):
        g.replay()
        assert torch.equal(out.cpu(), expected(x, 0.5, 11, i))


def test_empty(z):
    for shape in ((0, 8), (8, 0)):
        assert z.Dropout(0.5).apply(torch.zeros(shape, device="cuda")).shape == shape
