"""GPU: the balance of sequences so long that a lane has tens of thousands of tokens.

Equal rows give equal shares q, whose sum has a closed form; added one after the other in
32 bits each sum would be off in the same direction again and again.  The ways here: a
share (64 roundings), a run of at most 512 of a lane and at most 256 runs, 16 warps, 304
parts: under 1200 roundings, each by at most 2^-24 of the sum, as all terms are positive."""
import pytest
import torch

from gpu_util import load_lib, require_gpu

pytestmark = pytest.mark.gpu
LOSS = 1200 * 2.0 ** -24


@pytest.fixture(scope="module")
def z():
    require_gpu()
    load_lib()
    import lossless_bf16_exponent_split_gb300 as z
    return z


# tokens, how many sequences without tokens are behind them, experts, the one that all tokens choose
@pytest.mark.parametrize("tokens,others,experts,chosen", [
    (1 << 22, 305, 2, 0), (1 << 22, 305, 2, 1), (1 << 22, 305, 8, 0), (1 << 20, 400, 200, 3), (100_001, 304, 300, 7),
    (1 << 27, 0, 2, 0), (1 << 27, 0, 2, 1), (1 << 26, 3, 2, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_tokens_of_a_sequence(z, tokens, others, experts, chosen, score):
    row = torch.randn(experts, generator=torch.Generator().manual_seed(1))
    logits = row.cuda().repeat(tokens, 1)
    idx = torch.full((tokens, 1), chosen, dtype=torch.int32, device="cuda")
    seq = torch.tensor([0] + [tokens] * (others + 1), dtype=torch.int32, device="cuda")
    got = z.Moe(experts, 1, score=score).balance(logits, idx, seq)
    q = torch.softmax(row.double(), 0) if score == "softmax" else torch.sigmoid(row.double()) / torch.sigmoid(row.double()).sum()
    want = experts * float(q[chosen])
    assert abs(float(got.loss) - want) <= LOSS * want
    assert got.tokens.tolist() == [tokens] + [0] * others + [1]
    assert int(got.counts[0, chosen]) == tokens == int(got.counts.sum())
