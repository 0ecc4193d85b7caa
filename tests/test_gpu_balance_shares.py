"""GPU: how far a share is from its value in 64 bits.

One token that names one expert of E has the loss E q.  With d the distance to the row's
largest logit (sigmoid: the logit's size) q is off by at most, in units of 2^-24: 1.5 d for the
rounded difference, the product with the rounded log2 e and that; 4 for the exponential, the same
again with 1.5 / e for the sum's terms (their d weighted by themselves), 21 for a sum of 16 a lane and 5 halvings, 4 for
the reciprocal and the product, 6 for the loss: under (2 d + 48), and the header has 4 (d + 16)."""
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


@pytest.mark.parametrize("experts", [2, 64, 100, 512])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_share_of_one_token(z, experts, score):
    g = torch.Generator().manual_seed(experts)
    moe = z.Moe(experts, 1, score=score)
    for i in range(200):
        spread = 20.0 * torch.rand(1, generator=g)
        row = torch.randn(experts, generator=g) * spread + torch.randn(1, generator=g)
        e = int(torch.randint(0, experts, (1,), generator=g))
        got = moe.balance(row[None].cuda(), torch.tensor([[e]], dtype=torch.int32, device="cuda"))
        l = row.double()
        d = l.max() - l[e] if score == "softmax" else l[e].abs()
        q = torch.softmax(l, 0) if score == "softmax" else torch.sigmoid(l) / torch.sigmoid(l).sum()
        want = experts * float(q[e])
        if want / experts < 2.0 ** -120:
            continue  # its score may read as none
        assert abs(float(got.loss) - want) <= (float(d) + 16) * 2.0 ** -22 * want, (i, e)
