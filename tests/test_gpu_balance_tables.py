"""GPU: the balance over tables of sequences that do not cover all tokens, or run backwards."""
import pytest
import torch

import norm_ref as ref
from gpu_util import load_lib, require_gpu
from test_gpu_balance import LOSS, close, inputs

pytestmark = pytest.mark.gpu
F = torch.float32


@pytest.fixture(scope="module")
def z():
    require_gpu()
    load_lib()
    import lossless_bf16_exponent_split_gb300 as z
    return z


def gradient(z, moe, l, idx, got, seq, fill):
    """balance_backward into a buffer that holds `fill`."""
    out = torch.full_like(l, fill)
    st = z.zccl_balance_backward(moe.config, l.data_ptr(), z.F32, l.shape[1], idx.data_ptr(), l.shape[0], seq.data_ptr(),
                                 seq.shape[0] - 1, got.counts.data_ptr(), got.tokens.data_ptr(), 1.0, None, out.data_ptr(),
                                 l.shape[1], 0, torch.cuda.current_stream().cuda_stream)
    assert st == z.OK
    return out


# the first sequence's first token, sequences, the tokens of each, tokens behind them
@pytest.mark.parametrize("first,sequences,each,behind", [
    (7, 1, 93, 0), (64, 3, 100, 30), (1, 304, 5, 1), (1000, 2, 0, 0), (5, 305, 3, 0), (2000, 400, 2, 0), (300, 400, 2, 5000),
    (70000, 305, 1, 1), (1, 305, 0, 0), (2, 310, 0, 3)])
def test_tokens_before_the_first_and_behind_the_last(z, first, sequences, each, behind):
    """They do not count, and every row of the gradient is written."""
    tokens = first + sequences * each + behind
    l, idx = inputs(tokens, 12, 3, F)
    bounds = [first + s * each for s in range(sequences + 1)]
    moe, seq = z.Moe(12, 3), torch.tensor(bounds, dtype=torch.int32, device="cuda")
    loss, counts, live, grad, mag = ref.balance(l, idx, bounds, "softmax")
    got = moe.balance(l, idx, seq)
    assert torch.equal(got.counts.cpu(), counts) and torch.equal(got.tokens.cpu(), live)
    assert abs(float(got.loss) - loss) <= LOSS * abs(loss)
    have = gradient(z, moe, l, idx, got, seq, 7.0)
    close(have, grad, mag)
    assert bool((have[:first] == 0).all()) and bool((have[tokens - behind:] == 0).all())
    base = torch.randn_like(l)
    out = moe.balance_backward(l, idx, got, seq, out=base.clone())
    close(out, base.double().cpu() + grad, base.double().cpu().abs() + mag)
    assert torch.equal(out[:first], base[:first]) and torch.equal(out[tokens - behind:], base[tokens - behind:])
