"""GPU: dispatch on both sides of its choice of kernels, with rows long enough
that several CTAs share a counted tile."""
import numpy as np
import pytest
import torch

import moe_ref as ref
from gpu_util import load_lib, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def z():
    require_gpu()
    load_lib()
    import lossless_bf16_exponent_split_gb300 as z
    return z


@pytest.mark.parametrize("t,e,k,h", [
    (12288, 7, 2, 520), (12289, 7, 2, 520), (1536, 64, 16, 1000), (1537, 64, 16, 1000), (30000, 512, 1, 264), (1500, 40, 20, 2048),
    (300007, 3, 1, 8), (160000, 90, 3, 16),
])
def test_dispatch(z, t, e, k, h):
    rng = np.random.default_rng(t + h)
    idx = np.minimum((rng.random((t, k)) ** 2 * e).astype(np.int32), e - 1)
    idx[rng.random((t, k)) < 0.05] = -1
    x = torch.randint(-32768, 32768, (t, h), dtype=torch.int16, generator=torch.Generator("cuda").manual_seed(t), device="cuda")
    moe = z.Moe(e, k)
    pos, counts, offsets, order = ref.places(idx, e)
    total = int(offsets[-1])
    want = x[torch.from_numpy(order // k).cuda().long()]
    want[total:] = 0
    for _ in range(2):
        d = moe.dispatch(x.view(torch.bfloat16), torch.from_numpy(idx).cuda())
        assert np.array_equal(d.pos.cpu().numpy(), pos)
        assert np.array_equal(d.counts.cpu().numpy(), counts)
        assert np.array_equal(d.offsets.cpu().numpy(), offsets)
        assert torch.equal(d.rows.view(torch.int16), want)
